// rda_mla_decode_q4.hip -- absorbed latent attention over a paged latent cache
// in 4 bits: for a query row q and the cached rows c_j that it sees,
//   s_j = scale q . c_j,  m = some reference,  p_j = exp(s_j - m),
//   o = sum_j p_j c_j[0:512] / sum_j p_j,  lse = m + log sum_j p_j.
//
// A cached row is 400 bytes and is read once for 32 or 64 query rows, so one
// token of 32 heads is a matter of bytes, several tokens or a prefix that all
// share one of products (2176 flop a cached row and query row).
//
// Scores.  The codes enter the matrix instruction as they lie in LDS: it takes
// 4-bit operands with a scale byte per 32 values, and a 16-byte granule is one
// lane's share.  Its other operand has 8 bits at most, so a query is hi + lo, each
// e4m3 with a scale per 32 channels: 4 + 4 significant bits, as many as bf16 has.  The
// two products cost what one of bf16 over unpacked rows would, and nothing is unpacked
// for them.  The 64 shared channels are bf16 products.
// The instruction adds eight products at a time, each cut towards zero at 2^-13 of
// the power of two of the largest (and the eights' sums to 24 bits), so what a part
// holds must not lie too far below its largest: see stage_query.
// Values.  Probabilities are rounded to bf16 (once, off by 2^-8 at most) and the
// codes unpacked to bf16 (exact; each value once a workgroup, into its wave's own
// LDS), since the product runs over rows and scales go with channels: the probability
// would have to carry every group's scale.  Sums O^T, 32 channels by 32 query rows
// a block, stay in placed accumulation registers.
// Softmax.  The reference of a row moves only when the row outgrows it by 2^8, so
// the sums are hardly ever rescaled; scores, probabilities' sums and outputs are
// held in fp32.
//
// A workgroup has a wave per 16 query rows and half a tile of 32 cached rows for the
// scores, and each wave sums 128 or 64 channels of all its query rows.  Tile
// i + 1's scores run beside tile i's values, with one barrier a tile.  Tiles come by
// LDS-DMA in a ring of 4 or 8; their addresses are looked up 64 tiles at a time, one a
// lane.  The tiles of all sequences are one line that is cut into equal shares on
// the device (walk_sequences), and what is cut is joined by a second kernel.
//
// Bound by: the waits between those stages.  Of 3700 cycles for two tiles of a CU's
// two workgroups 1090 are matrix instructions and 1650 LDS transfers (an unpacked
// granule costs 13 cycles to write and 2 a row to read transposed).
//   256 sequences of 512 to 8192 rows, 32 query rows: 132 us of which the joining takes
//     10; 474 MB, 3.6 TB/s (78 us at 6.1)
//   32 of them, 96 query rows: 64 us
//   12288 query rows behind 16384 shared rows: 453 us, 985 TFLOP/s
//   one sequence of 131072 rows: 38 us; of 777: 16
// Not faster: values read transposed as codes with the scale as an exponent added to
// the probability (158.6 us for the first case and 577 for the third, both 10 %
// slower: 220 ordinary instructions a wave and tile for 160); 128 query rows a
// workgroup with one wave a SIMD and 256 sums (32 x 3 tokens 95 us for 79);
// half of the waves unpacking at the other end of a tile (82 for 79); sums stored
// past the caches (160 for 156).
#include <type_traits>

#include "rda_mla_q4.h"

namespace rda {
namespace {

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;                        // cached rows per tile
constexpr int kTileBytes = kTile * kQ4Row;       // 12800
constexpr int kJoinThreads = 256;
// How many waves join a query row: 16 times 8 or 4 slices of channels up to the first
// and second number of rows (256 workgroups each), 4 up to the third, else one.  64 rows
// with 256 pieces 40 us in all for 45.5 with four waves (with 31 pieces 19.4 for 17.6),
// but 128 rows 22.4 for 19.8; workgroups of 1024 threads are slow to start, a second one
// on each CU (64 rows in 8 slices) costs 2 us.  256 rows with 128 pieces 37 us for 43
// with one wave, 512 rows with 64 pieces equal, 2048 rows with 2 pieces 40 for 37.
constexpr int kEightRows = 32, kWideRows = kQ4FewRows, kFourRows = 512;
// What a unit costs a workgroup beside its tiles (queries in, sums out: 7 to 8 us), in
// tiles.  60 sequences of 500 to 4000 rows, 2 tokens: 49 us at 3, 46.8 at 6, 44.4 at 8;
// 256 of one token 147, 143 and 146.  (The limits that the caller checks count 6 for each
// 32 query rows.)
template <int kRW>
constexpr int kPieceTiles = kRW == 2 ? 8 : 6;
// Shares of fewer tiles than this for two workgroups a CU are made twice as long for
// one: half the pieces to write and join, but no second workgroup to fill a tile's
// waits.  65536 rows (4 tiles) 32.6 us for 35.7, 16 x 2048 27.4 for 31.8; 131072 (8)
// 41.8 either way; 64 of 1000 and 3000 rows (8) 42.3 for 39.5.
constexpr int kBothTiles = 6;

// A workgroup of 32 kRW query rows: 4 kRW waves.  One of 32 rows leaves room for a
// second on its CU; one of 64 reads a tile once for twice the rows.
template <int kRW>
struct Shape {
    static constexpr int kWaves = 4 * kRW, kThreads = 64 * kWaves;
    static constexpr int kRowWaves = 2 * kRW, kKeyWaves = 2;        // of 16 query rows, 16 cached rows each
    static constexpr int kFetchRows = kTile / 4;                    // waves 0 .. 3 fetch a tile
    static constexpr int kChannels = kMlaLatent / kWaves;           // that a wave sums
    static constexpr int kBlocks = kChannels / 32;
    static constexpr int kValRows = 16 * kRW;                       // rows that a wave unpacks at a time
    static constexpr int kValRow = kChannels * 2, kValBytes = kValRows * kValRow;
};

template <int kRW>
struct Lds {
    static constexpr int kBuf = 4 * kRW;   // tiles in flight or in use
    unsigned char tile[kBuf][kTileBytes];   // (the last two and what follows: queries on their way in)
    unsigned char val[Shape<kRW>::kWaves][Shape<kRW>::kValBytes];   // a wave's own: unpacked values
    u32x4 p[2][kRW][kTile / 16][64];   // probabilities: [32 query rows][16 cached rows][lane]
    float top[Shape<kRW>::kWaves][16];
    float l[Shape<kRW>::kWaves][16];
    uint32_t qscale[kRW * 32][kQ4Groups / 4];
    float mu[kRW * 32];
    float factor[kRW * 32];
    int moved[2];
    int scan[2 * Shape<kRW>::kWaves];
    int unit, first;
};

template <int kN, typename F>
__device__ __forceinline__ void each(F f) {
    if constexpr (kN > 0) {
        each<kN - 1>(f);
        f(std::integral_constant<int, kN - 1>{});
    }
}

// Largest of x over the lanes l ^ 16, l ^ 32, and their sum.
__device__ __forceinline__ float max_over_quarters(float x) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ uint32_t umax_over_quarters(uint32_t x) {
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max(uint32_t(r[0]), uint32_t(r[1]));
    r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return max(uint32_t(r[0]), uint32_t(r[1]));
}
__device__ __forceinline__ float sum_over_quarters(float x) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ uint32_t lds_read4(uint32_t a) {
    typedef __attribute__((address_space(3))) uint32_t lds_u32;
    return *(const lds_u32*)(lds_char*)uintptr_t(a);
}
__device__ __forceinline__ u32x4 lds_read_u4(uint32_t a) {
    return *(const lds_u32x4*)(lds_char*)uintptr_t(a);
}
__device__ __forceinline__ void lds_write_u2(uint32_t a, u32x2 x) {
    typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
    *(lds_u32x2*)(lds_char*)uintptr_t(a) = x;
}
__device__ __forceinline__ void lds_write_u4(uint32_t a, u32x4 x) {
    *(lds_u32x4*)(lds_char*)uintptr_t(a) = x;
}

// Row r of unpacked values (256 or 128 bytes) keeps 16-byte granule j at
// j ^ val_swz(r): eight rows written at one granule, and the rows and granules
// that a transposing read touches at a time, fall on distinct banks.
template <int kRow>
__device__ __forceinline__ int val_swz(int r) {
    return (r >> 1 & 1) * (kRow == 256 ? 10 : 4) | (r & 1) * (kRow == 256 ? 4 : 2) | (r >> 2 & 1);
}

__device__ __forceinline__ int clamp_len(const MlaDecodeArgs& A, int b) {
    const int64_t most = int64_t(A.table_width) << A.page_shift;
    const int n = A.kv_lens[b];
    return A.num_pages > 0 && n > 0 ? int(n < most ? n : most) : 0;
}

struct Source {
    const int32_t* table;
    int len;
};

// Where a piece's sums go: the outputs, or a slot of partial sums.
struct Sink {
    bool final;
    int64_t row0;      // first query row of the unit's block (outputs)
    int first_row;     // the same, from the sequence's first query row
    int rows;          // query rows of the unit
    float* part;       // [unit rows][512]
    float* ml;         // [unit rows][2]
};

// A query row block of 16 as the scores' second operand.
struct Query {
    i32x8 hi[4], lo[4];
    bf16x8 pe[2];
    uint32_t hi_scale, lo_scale;   // scale bytes of the lane's groups
};

// Query rows as pairs of 8-bit values into LDS at `at` (hi, then lo: 512 bytes a
// row, 16-byte granule j at j ^ (row & 15)) and hi's scale bytes, one for each 32
// channels, into `scales`: kStaged rows a wave, eight values a lane.
//
// The largest value of 32 lands in [1.94, 3.88) of hi's scale, where 8-bit floats end
// in steps of 2^-9, so hi is a whole multiple of 2^-9 and no more than 3.75.  With codes,
// multiples of 1/2 up to 6, its products end at 2^-10 and their powers of two are 2^3 at
// most: 2^-13 apart, so they are added whole.  What hi leaves is 2^-3 at most, 256 in
// lo's scale, whose products are cut at 2^-3 of it (2^-14 of hi's) or below.  A
// value of 1/64 or more of the largest is thus held and multiplied exactly; a smaller one
// is off by what 4 bits of 2^-10 leave (2^-15 of hi's scale) and its products by the cut
// (2^-14 of hi's, times the unit of the codes).
// With one scale a row and the largest at [128, 256), which holds all but 2^-22 of
// it, hi's own products were cut: normal queries' scores 4e-5 off (root mean square; now
// 1e-5), 5e-4 where channels differ widely (now 1.7e-4).
constexpr int kStaged = 8;
constexpr int kLoBelow = 11;           // lo's scale byte is that much below hi's
constexpr int kQueryLeast = 16;          // (what lower scales would hold is subnormal in 32 bits)
template <int kRW>
__device__ __forceinline__ void stage_query(const u32x4* x, uint32_t at, uint32_t (*scales)[kQ4Groups / 4]) {
    static_assert(kStaged * Shape<kRW>::kWaves == 32 * kRW, "all rows");
    const int w = wave_id(), l = here(threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < kStaged; ++i) {
        const int row = kStaged * w + i;
        u16x2 most = {};
#pragma unroll
        for (int d = 0; d < 4; ++d)
            most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, x[i][d] & 0x7fff7fffu));
        uint32_t top = max(uint32_t(most[0]), uint32_t(most[1]));   // of the group's four lanes
        top = max(top, uint32_t(__builtin_amdgcn_update_dpp(0, int(top), 0xB1, 0xF, 0xF, false)));
        top = max(top, uint32_t(__builtin_amdgcn_update_dpp(0, int(top), 0x4E, 0xF, 0xF, false)));
        // (from 1.9375 on it counts as the next power: hi would round up to it)
        const uint32_t sh = top >= 0x7f80u ? kQ4Bad : max(int((top + 8) >> 7) - 1, kQueryLeast);
        const float fh = q4_scale(sh), fl = q4_scale(sh - kLoBelow);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int d = 0; d < 2; ++d) {   // four values a dword
            s16x2 y = {}, z = {};
            const uint32_t a = x[i][2 * d], b = x[i][2 * d + 1];
            y = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(y, __builtin_bit_cast(bf16x2, a), fh, false);
            y = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(y, __builtin_bit_cast(bf16x2, b), fh, true);
            hi[d] = __builtin_bit_cast(uint32_t, y);
            const f32x2 ra = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi[d], fh, false);
            const f32x2 rb = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi[d], fh, true);
            z = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(
                z, __uint_as_float(a << 16) - ra[0], __uint_as_float(a & 0xffff0000u) - ra[1], fl, false);
            z = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(
                z, __uint_as_float(b << 16) - rb[0], __uint_as_float(b & 0xffff0000u) - rb[1], fl, true);
            lo[d] = __builtin_bit_cast(uint32_t, z);
        }
        const uint32_t to = at + row * 512 + 16 * ((l >> 1) ^ (row & 15)) + 8 * (l & 1);
        lds_write_u2(to, u32x2{hi[0], hi[1]});
        lds_write_u2(to + 32 * kRW * 512, u32x2{lo[0], lo[1]});
        if ((l & 3) == 0) reinterpret_cast<unsigned char*>(scales[row])[l >> 2] = static_cast<unsigned char>(sh);
    }
}

// Its 16 rows of them as a wave's operands.
template <int kRW>
__device__ __forceinline__ void take_query(Query& Q, uint32_t at, const uint32_t (*scales)[kQ4Groups / 4], int row,
                                           int t) {
    auto sixteen = [&](int part, int g) {   // 16 bytes
        return lds_read_u4(at + (32 * kRW * part + row) * 512 + 16 * (g ^ (row & 15)));
    };
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int g = 2 * (4 * (t >> 1) + m) + (t & 1);
        const u32x4 a = sixteen(0, g), b = sixteen(0, g + 16), c = sixteen(1, g), d = sixteen(1, g + 16);
        Q.hi[m] = i32x8{int(a[0]), int(a[1]), int(a[2]), int(a[3]), int(b[0]), int(b[1]), int(b[2]), int(b[3])};
        Q.lo[m] = i32x8{int(c[0]), int(c[1]), int(c[2]), int(c[3]), int(d[0]), int(d[1]), int(d[2]), int(d[3])};
    }
    Q.hi_scale = scales[row][t];
    Q.lo_scale = Q.hi_scale - uint32_t(kLoBelow) * 0x01010101u;
}

// The reference of a row that has seen no score: any score outgrows it, however small
// the scale is ((score + infinity) c is infinite for every c > 0, subnormal ones too),
// and a row of masked places alone does not (NaN compares as no).
constexpr float kNone = -INFINITY;

// One piece: tiles [t0, t1) of a source for 32 kRW query rows.
template <int kRW, bool kCausal>
__device__ __forceinline__ void piece(const MlaDecodeArgs& A, Lds<kRW>& lds, const Source& src, int t0,
                                      int t1, const Sink& sink, int& turn) {
    typedef Shape<kRW> S;
    constexpr int kBuf = Lds<kRW>::kBuf, kBlocks = S::kBlocks, kValRow = S::kValRow;
    const int w = wave_id(), l = threadIdx.x & 63;
    const int rw = w % S::kRowWaves, kw = w / S::kRowWaves;
    const int c16 = l & 15, t = l >> 4, c32 = l & 31, g = l >> 5;
    const int end = min(src.len, t1 * kTile);
    const float c = A.scale * kLog2e;
    const uint32_t tiles = lds_addr(&lds.tile[0][0]);
    const uint32_t val = lds_addr(&lds.val[w][0]);

    // lane j: where this wave's rows of tile rows_from + j lie
    const char* rows = nullptr;
    int rows_from = t0;
    auto row_of = [&]() { return (rows_from + l) * kTile + S::kFetchRows * w; };
    auto page_of = [&](int k) { return src.table[k < src.len ? k >> A.page_shift : 0]; };
    auto place = [&](int k, int page) {
        rows = reinterpret_cast<const char*>(A.cache) +
               int64_t(min(max(page, 0), A.num_pages - 1)) * A.page_stride +
               (k & ((1 << A.page_shift) - 1)) * kQ4Row;
    };
    const uint32_t lane16 = 16 * l;
    auto issue = [&](int tile) {
        if (S::kWaves > 4 && w >= 4) return;
        if (tile - rows_from == 64) {
            rows_from = tile;
            place(row_of(), page_of(row_of()));
        }
        const int j = tile - rows_from;
        const uint64_t r = reinterpret_cast<uint64_t>(rows);
        const char* const from = reinterpret_cast<const char*>(
            uint64_t(uint32_t(__builtin_amdgcn_readlane(int(r >> 32), j))) << 32 |
            uint32_t(__builtin_amdgcn_readlane(int(r), j)));
        const int valid = end - (tile * kTile + S::kFetchRows * w);
        const uint32_t to = tiles + (tile - t0) % kBuf * kTileBytes + w * S::kFetchRows * kQ4Row;
        // (a sequence's rows pass the caches by where one block of query rows reads them,
        // not where several do: 32 x 3 tokens 64.4 us for 65.1)
        if (__builtin_expect(valid >= S::kFetchRows, 1)) {
            if (kCausal && (kRW == 1 || A.row_blocks == 1)) q4_fetch_rows<true>(from, lane16, to);
            else q4_fetch_rows<false>(from, lane16, to);
        } else if (valid <= 0) q4_fetch_rows<false>(kQ4Zeros, lane16, to);
        else q4_fetch_some(from, valid, l, to);
    };
    // Page numbers and queries come in at the same time, then two tiles beside which
    // the queries are converted (32 x 3 tokens 66.5 us for 68.6 with the queries after
    // the tiles, 60 x 40 heads 44.6 for 46.5).
    int page = 0;
    if (S::kWaves == 4 || w < 4) page = page_of(row_of());
    Query q;
    float m = kNone, mu = 0.f, lsum = 0.f;
    const int qrow = min(16 * rw + c16, sink.rows - 1);
    u32x4 x[kStaged];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kStaged; ++i)
        x[i] = *reinterpret_cast<const u32x4*>(
            A.q + (sink.row0 + min(kStaged * w + i, sink.rows - 1)) * kMlaRow + 8 * l);
#pragma unroll
    for (int n = 0; n < 2; ++n)
        q.pe[n] = __builtin_bit_cast(
            bf16x8, *reinterpret_cast<const u32x4*>(A.q + (sink.row0 + qrow) * kMlaRow + kMlaLatent + 32 * n + 8 * t));
    __builtin_amdgcn_sched_barrier(0);
    place(row_of(), page);
#pragma unroll 1
    for (int d = 0; d < 2; ++d) issue(t0 + d);
    {
        static_assert(2 * kTileBytes + sizeof(lds.val) + sizeof(lds.p) >= 32 * kRW * 1024, "room for the queries");
        const uint32_t at = tiles + (kBuf - 2) * kTileBytes;
        stage_query<kRW>(x, at, lds.qscale);
#pragma unroll 1
        for (int d = 2; d < kBuf - 2; ++d) issue(t0 + d);
        raw_barrier();
        take_query<kRW>(q, at, lds.qscale, 16 * rw + c16, t);
        raw_barrier();
        issue(t0 + kBuf - 2);
    }
    // (rows from `end` on, which belong to others or to nobody, are behind every limit)
    const int limit = min(end, kCausal ? src.len - (A.tokens - 1 - (sink.first_row + qrow) / A.heads) : src.len);
    const int all_see = min(end, kCausal ? src.len - (A.tokens - 1) : src.len);
    // block kBlocks rb + b: 32 query rows by 32 channels
    static_assert(kRW * kBlocks == 4, "the accumulation registers");
    each<64>([](auto x) { q4_acc_clear<decltype(x)::value>(); });

    // this lane's addresses, from a tile's start
    const uint32_t krow = (kw * 16 + c16) * kQ4Row;                          // the row it scores
    const int urow = l % S::kValRows, ugroup = l / S::kValRows;              // what it unpacks
    const uint32_t drow = urow * kQ4Row + S::kChannels / 2 * w + 16 * ugroup;
    const int dbyte = S::kChannels / kQ4Group * w;
    const uint32_t dscale = urow * kQ4Row + kQ4ScaleAt + (dbyte & ~3);
    const int dshift = 8 * ((dbyte & 3) + ugroup);
    const uint32_t vput = val + urow * kValRow + 16 * (4 * ugroup ^ val_swz<kValRow>(urow));
    const int vr = 8 * g + (c16 >> 2), vlow = 2 * (t & 1) + ((c16 >> 1) & 1);
    uint32_t vget[2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
        vget[n] = val + (vr + 4 * n) * kValRow + 16 * (vlow ^ val_swz<kValRow>(vr + 4 * n)) + 8 * (c16 & 1);
    const uint32_t pput = lds_addr(&lds.p[0][rw >> 1][kw][16 * (rw & 1) + c16 + 32 * (t >> 1)]) + 8 * (t & 1);
    const uint32_t pget = lds_addr(&lds.p[0][0][0][l]);

    // A tile's stages.  Scores of 16 cached rows: operands by halves, products.
    f32x4 hi, lo;   // two chains: a product waits for the one before
    uint32_t kscale;
    u32x4 k4[4];
    bf16x8 pe[2];
    auto read_scale = [&](uint32_t tile) { kscale = lds_read4(tile + krow + kQ4ScaleAt + 4 * t); };
    auto read_rows = [&](uint32_t tile, int half) {
#pragma unroll
        for (int n = 2 * half; n < 2 * half + 2; ++n) k4[n] = lds_read_u4(tile + krow + 64 * t + 16 * n);
    };
    auto read_pe = [&](uint32_t tile) {
#pragma unroll
        for (int n = 0; n < 2; ++n) pe[n] = lds_read16(tile + krow + kQ4PeAt + 64 * n + 16 * t);
    };
    auto score = [&](auto nn) {
        constexpr int n = decltype(nn)::value;
        q4_score<n>(hi, k4[n], q.hi[n], kscale, q.hi_scale);
        q4_score<n>(lo, k4[n], q.lo[n], kscale, q.lo_scale);
    };
    auto score_pe = [&]() {
        q4_score_pe(hi, pe[0], q.pe[0]);
        q4_score_pe(lo, pe[1], q.pe[1]);
    };
    auto scores = [&]() { each<4>(score); };
    // Values: a lane unpacks a group of 32 channels of a row.
    constexpr int kParts = kTile / S::kValRows;
    u32x4 codes[kParts];
    uint32_t scales[kParts];
    auto read_codes = [&](uint32_t tile) {
#pragma unroll
        for (int x = 0; x < kParts; ++x) {
            codes[x] = lds_read_u4(tile + drow + x * S::kValRows * kQ4Row);
            scales[x] = lds_read4(tile + dscale + x * S::kValRows * kQ4Row);
        }
    };
    float unit;
    auto unpack_scale = [&](int x) {
        // NaN groups are left out here: they have made the scores of all who see
        // them NaN, and no others may meet them as 0 x NaN
        const uint32_t sb = (scales[x] >> dshift) & 255;
        unit = q4_scale(sb == kQ4Bad ? 0 : sb);
    };
    auto unpack = [&](int x, int j) { lds_write_u4(vput ^ (16 * j), q4_eight(codes[x][j], unit)); };
    auto unpack_all = [&](int x) {
        unpack_scale(x);
#pragma unroll
        for (int j = 0; j < 4; ++j) unpack(x, j);
    };
    // The products of 16 cached rows with their probabilities.
    bf16x8 v[kBlocks], pr[kRW];
    auto read_p = [&](int i, int step) {
#pragma unroll
        for (int rb = 0; rb < kRW; ++rb)
            pr[rb] = lds_read16(pget + (i & 1) * sizeof(lds.p[0]) + rb * sizeof(lds.p[0][0]) +
                                step * sizeof(lds.p[0][0][0]));
    };
    auto read_values = [&](int step) {
        const uint32_t at = kParts == 1 ? step * 16 * kValRow : 0;
        const uint32_t get[2] = {uint32_t(here(int(vget[0]))), uint32_t(here(int(vget[1])))};
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const u32x2 y = lds_read_tr8((get[0] ^ (64 * b)) + at), z = lds_read_tr8((get[1] ^ (64 * b)) + at);
            v[b] = __builtin_bit_cast(bf16x8, u32x4{y[0], y[1], z[0], z[1]});
        }
    };
    auto add_values = [&](auto nn) {   // the n-th of four
        constexpr int n = decltype(nn)::value, b = n / kRW, rb = n % kRW;
        q4_acc_product<kBlocks * rb + b>(v[b], pr[rb]);
    };
    // Softmax of tile i's scores against the reference that stands.
    f32x4 s;
    float top, before;
    auto store_p = [&](int i) {
        f32x4 e;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            e[x] = __builtin_amdgcn_exp2f(fmaf(s[x], c, -mu));
            lsum += e[x];
        }
        lds_write_u2(pput + (i & 1) * sizeof(lds.p[0]), u32x2{pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3])});
    };
    auto mask = [&](int i) {
        const int k0 = (t0 + i) * kTile;
        q4_score_done(hi, lo);
        s = hi + lo;
        if (__builtin_expect(k0 + kTile > all_see, 0)) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (k0 + 16 * kw + 4 * t + x >= limit) s[x] = -INFINITY;
        }
    };
    // The reference moves only when a row outgrows it by 2^8: the probabilities go
    // out against the one that stands, and again where it moves.
    auto probabilities = [&](int i) {
        before = lsum;
        store_p(i);
    };
    auto look = [&](int i) {
        top = max_over_quarters(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])));
        if (__any((top - m) * c > 8.f)) lds.moved[i & 1] = turn + i;
    };
    auto fence = [] { __builtin_amdgcn_sched_barrier(0); };

    wait_vm<(kBuf - 2) * kQ4Fetch>();
    raw_barrier();
    read_scale(tiles);
    read_rows(tiles, 0);
    read_rows(tiles, 1);
    read_pe(tiles);
    scores();
    score_pe();
    read_codes(tiles);
    mask(0);
    probabilities(0);
    look(0);
    unpack_all(0);
    const int n_tiles = t1 - t0;
#pragma unroll 1
    for (int i = 0; i < n_tiles; ++i) {
        // (two workgroups of a CU take turns: left alone the older one goes first, and
        // the younger ends 23 of 108 us later)
        if constexpr (kRW == 1) {
            if ((i ^ (blockIdx.x >> 8)) & 1) __builtin_amdgcn_s_setprio(1);
            else __builtin_amdgcn_s_setprio(0);
        }
        wait_vm<(kBuf - 3) * kQ4Fetch>();   // this wave's part of the next tile
        raw_barrier();                      // everyone's; the tile before is read
        const uint32_t next = tiles + ((i + 1) % kBuf) * kTileBytes;
        const int moved = lds.moved[i & 1];
        // The scores of the next tile (none behind the last) beside this one's sums,
        // in this order: LDS reads well before their use, few operands at a time.
        read_values(0);
        read_scale(next);
        read_rows(next, 0);
        fence();
        if (__builtin_expect(__builtin_amdgcn_readfirstlane(moved) == turn + i, 0)) {
            if (t == 0) lds.top[w][c16] = top;
            raw_barrier();
            float mn = fmaxf(m, top);
#pragma unroll
            for (int k = 0; k < S::kKeyWaves; ++k) mn = fmaxf(mn, lds.top[k * S::kRowWaves + rw][c16]);
            // (a row that has not outgrown its own keeps it: its result does not
            // depend on the rows beside it)
            if (!((mn - m) * c > 8.f)) mn = m;
            const float mun = mn == kNone ? 0.f : mn * c;
            const float a = m == kNone ? 0.f : __builtin_amdgcn_exp2f(mu - mun);
            m = mn;
            mu = mun;
            lsum = before * a;
            if (kw == 0 && t == 0) lds.factor[16 * rw + c16] = a;
            store_p(i);
            raw_barrier();
            float f[kRW];
#pragma unroll
            for (int rb = 0; rb < kRW; ++rb) f[rb] = lds.factor[32 * rb + c32];
            q4_acc_settle();
            each<64>([&](auto x) { q4_acc_scale<decltype(x)::value>(f[decltype(x)::value / (16 * kBlocks)]); });
        }
        read_p(i, 0);
        fence();
        // (matrix instructions run beside the ordinary ones that follow them)
        if constexpr (kParts > 1) unpack_scale(1);
        each<4>([&](auto nn) {
            add_values(nn);
            if constexpr (kParts > 1) unpack(1, decltype(nn)::value);
            fence();
        });
        read_rows(next, 1);
        read_p(i, 1);
        read_values(1);
        read_pe(next);
        fence();
        scores();
        score_pe();
        issue(t0 + i + kBuf - 1);
        read_codes(next);
        fence();
        add_values(std::integral_constant<int, 0>{});
        fence();
        mask(i + 1);
        fence();
        add_values(std::integral_constant<int, 1>{});
        fence();
        probabilities(i + 1);
        fence();
        add_values(std::integral_constant<int, 2>{});
        fence();
        look(i + 1);
        unpack_scale(0);
        fence();
        add_values(std::integral_constant<int, 3>{});
#pragma unroll
        for (int j = 0; j < 4; ++j) unpack(0, j);
    }
    wait_vm<0>();   // the tiles behind the last: nothing may land later
    raw_barrier();
    {
        // (addresses computed here: kept from the start they would crowd out the loop)
        const int l = here(threadIdx.x & 63), c16 = l & 15, t = l >> 4, c32 = l & 31, g = l >> 5;
        lsum = sum_over_quarters(lsum);
        if (t == 0) {
            lds.l[w][c16] = lsum;
            if (kw == 0) lds.mu[16 * rw + c16] = m == kNone ? -INFINITY : mu;
        }
        raw_barrier();
        q4_acc_settle();
        each<kRW>([&](auto rr) {
            constexpr int rb = decltype(rr)::value;
            float total = 0.f;
#pragma unroll
            for (int k = 0; k < S::kKeyWaves; ++k) total += lds.l[k * S::kRowWaves + 2 * rb + (c32 >> 4)][c16];
            const int lr = 32 * rb + c32;
            if (w == rb && g == 0 && lr < sink.rows) {
                const float x = lds.mu[lr];
                if (!sink.final) *reinterpret_cast<f32x2*>(sink.ml + 2 * lr) = f32x2{x, total};
                else if (A.lse) A.lse[sink.row0 + lr] = total == 0.f ? -INFINITY : fmaf(x, kLn2, logf(total));
            }
            const float inv = !sink.final ? 1.f : total == 0.f ? 0.f : 1.f / total;
            // 32 channels at a time by way of LDS, so that they leave row by row
            each<kBlocks>([&](auto bb) {
                constexpr int b = decltype(bb)::value;
                each<4>([&](auto xx) {
                    constexpr int x = decltype(xx)::value, r = 16 * (kBlocks * rb + b) + 4 * x;
                    const f32x4 y = {q4_acc_get<r>() * inv, q4_acc_get<r + 1>() * inv, q4_acc_get<r + 2>() * inv,
                                     q4_acc_get<r + 3>() * inv};
                    lds_write_u4(val + c32 * 128 + 16 * ((2 * x + g) ^ (c32 & 7)), __builtin_bit_cast(u32x4, y));
                });
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int r = 8 * x + (l >> 3), row = 32 * rb + r;
                    const f32x4 y = __builtin_bit_cast(
                        f32x4, lds_read_u4(val + r * 128 + 16 * ((l & 7) ^ (r & 7))));
                    if (row >= sink.rows) continue;
                    const int ch = S::kChannels * w + 32 * b + 4 * (l & 7);
                    if (sink.final)
                        *reinterpret_cast<u32x2*>(A.o + (sink.row0 + row) * kMlaLatent + ch) =
                            u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
                    else
                        *reinterpret_cast<f32x4*>(sink.part + size_t(row) * kMlaLatent + ch) = y;
                }
            });
        });
    }
    turn += n_tiles + 1;
    raw_barrier();   // the next piece writes what this one has read
}

// Sums of x over the lanes up to each.
__device__ __forceinline__ int scan64(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);   // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);   // row_shr:2
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);   // row_shr:4
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);   // row_shr:8
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);   // row_bcast:15 into rows 1 and 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);   // row_bcast:31 into rows 2 and 3
    return x;
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// Workgroup `wg` of those that share out the sequences' tiles.
template <int kRW>
__device__ __forceinline__ void walk_sequences(const MlaDecodeArgs& A, Lds<kRW>& lds, int wg, int workgroups) {
    constexpr int kThreads = Shape<kRW>::kThreads, kWaves = Shape<kRW>::kWaves;
    const int l = threadIdx.x & 63, w = wave_id();
    // up to 64 sequences: every wave for itself, a lane a sequence
    const bool few = A.batch <= 64;
    const int lane = few ? l : int(threadIdx.x);

    auto block_sum = [&](int x, int& before) {   // x over the lanes
        int s = scan64(x);
        if (few) {
            before = s - x;
            return __builtin_amdgcn_readlane(s, 63);
        }
        __syncthreads();
        if (l == 63) lds.scan[w] = s;
        __syncthreads();
        before = s - x;
        int total = 0;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            if (k < w) before += lds.scan[k];
            total += lds.scan[k];
        }
        return __builtin_amdgcn_readfirstlane(total);
    };
    auto tiles_at = [&](int b) { return b < A.batch ? tiles_of(clamp_len(A, b)) : 0; };
    // A unit's second and later pieces cost their workgroup nothing that it does not
    // pay anyway (queries in, sums out); a workgroup that goes on to another unit pays
    // again, as much as kPieceTiles tiles.  So the line that is cut into equal
    // shares holds that many places before each unit's tiles.
    const int n0 = tiles_at(lane);
    int head = kPieceTiles<kRW>, before0;
    auto places = [&](int n) { return n > 0 ? n + head : 0; };
    int x0 = places(n0);
    int total0 = block_sum(x0, before0);
    int total = total0;
    for (int b0 = kThreads; b0 < A.batch; b0 += kThreads) {
        int before;
        total += block_sum(places(tiles_at(b0 + int(threadIdx.x))), before);
    }
    total *= A.row_blocks;
    if (total == 0) return;
    const int units = A.batch * A.row_blocks;
    if (kRW == 1 && total < kBothTiles * workgroups) workgroups /= 2;
    int per = max((total + workgroups - 1) / workgroups, A.min_tiles);
    // Where the workgroups suffice for it none goes on to another unit: the units'
    // tiles are counted up to multiples of a share then, one as large as that line's
    // at most.  (Their sums are below four times the tiles' number.)
    bool apart = false;
    if (units <= workgroups && A.batch <= kThreads && total < 1 << 28) {
        int most = int(umax_over_quarters(dpp_umax16(uint32_t(n0)))), tiles;
        if (!few) {
            if (l == 0) lds.scan[kWaves + w] = most;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kWaves; ++k) most = max(most, lds.scan[kWaves + k]);
        }
        most = __builtin_amdgcn_readfirstlane(most);
        {
            int before;
            tiles = block_sum(n0, before);
        }
        int share = max(A.min_tiles, tiles * A.row_blocks / (workgroups - units / 2) + 1);
        for (int tries = 0; tries < 2 && !apart && share <= per; ++tries) {
            if (most <= share + 2) share = most;
            const int padded = (n0 + share - 1) / share * share;
            int before;
            const int sum = block_sum(padded, before);
            if (sum * A.row_blocks <= share * workgroups) {
                apart = true;
                per = share;
                head = 0;
                x0 = padded;
                before0 = before;
                total0 = sum;
                total = sum * A.row_blocks;
            }
            share += share / 8 + 1;
        }
    }
    if (int64_t(per) * wg >= total) return;
    int unit = 0, first = 0;
    const int begin = per * wg, end = begin + min(per, total - begin);
    for (int b0 = 0, seen = 0; b0 < A.batch && seen * A.row_blocks <= begin; b0 += kThreads) {
        const int b = b0 + lane;
        int x = x0, before = before0, sum = total0;
        if (b0 > 0) {
            x = places(tiles_at(b));
            sum = block_sum(x, before);
        }
        const int at = begin - (seen + before) * A.row_blocks;
        const bool mine = x > 0 && at >= 0 && at < x * A.row_blocks;
        if (few) {
            const int k = __builtin_ctzll(__ballot(mine));   // (one lane's share holds `begin`)
            const int n = __builtin_amdgcn_readlane(x, k), in = __builtin_amdgcn_readlane(at, k);
            unit = k * A.row_blocks + in / n;
            first = in % n;
        } else if (mine) {
            lds.unit = b * A.row_blocks + at / x;
            lds.first = at % x;
        }
        seen += sum;
    }
    if (!few) {
        __syncthreads();
        unit = lds.unit;
        first = lds.first;
    }
    unit = __builtin_amdgcn_readfirstlane(unit);
    first = __builtin_amdgcn_readfirstlane(first);

    const int unit_rows = A.tokens * A.heads;
    int at = begin, turn = 1;   // (turn: a number for each tile, for lds.moved)
    while (at < end) {
        const int b = unit / A.row_blocks, blk = unit - b * A.row_blocks;
        const int len = __builtin_amdgcn_readfirstlane(clamp_len(A, b));
        const int n = tiles_of(len);
        if (n == 0) {   // the joining kernel writes these rows
            ++unit;
            continue;
        }
        const int last = min(first + (end - at), n + head);
        const int t0 = max(first - head, 0), t1 = last - head;
        if (t0 < t1) {
            const bool whole = t0 == 0 && t1 == n;
            const int slot = t0 == 0 ? unit : units + wg;
            Sink sink;
            sink.final = whole && !A.prefix_len;
            sink.first_row = 32 * kRW * blk;
            sink.row0 = int64_t(b) * unit_rows + sink.first_row;
            sink.rows = min(32 * kRW, unit_rows - sink.first_row);
            sink.part = A.part + size_t(slot) * kMlaLatent * 32 * kRW;
            sink.ml = A.part_ml + size_t(slot) * 2 * 32 * kRW;
            if (t0 == 0 && threadIdx.x == 0) {
                // the workgroups that hold this unit's later pieces
                A.meta[2 * unit] = sink.final ? -1 : wg;
                A.meta[2 * unit + 1] = (at - first + n + head - 1) / per;
            }
            piece<kRW, true>(A, lds, Source{A.table + int64_t(b) * A.table_width, len}, t0, t1, sink, turn);
        }
        if (apart) break;
        at += last - first;
        first = 0;
        ++unit;
    }
}

// The prefix: every block of 32 kRW query rows walks all prefix rows.
template <int kRW>
__device__ __forceinline__ void walk_prefix(const MlaDecodeArgs& A, Lds<kRW>& lds, int wg) {
    const int rows = A.batch * A.tokens * A.heads;
    const int n = tiles_of(A.prefix_len), line = A.prefix_line;   // (its last line - n are none)
    const int total = A.prefix_units * line;
    int at = A.prefix_per * wg;
    const int end = at + min(A.prefix_per, total - at);
    int turn = 1;
    while (at < end) {
        const int unit = at / line, first = at - unit * line;
        const int last = min(first + (end - at), line);
        const int slot = first == 0 ? unit : A.prefix_units + wg;
        Sink sink;
        sink.final = false;
        sink.first_row = 0;
        sink.row0 = int64_t(unit) * 32 * kRW;
        sink.rows = min(32 * kRW, rows - unit * 32 * kRW);
        sink.part = A.pre_part + size_t(slot) * kMlaLatent * 32 * kRW;
        sink.ml = A.pre_ml + size_t(slot) * 2 * 32 * kRW;
        piece<kRW, false>(A, lds, Source{A.prefix_table, A.prefix_len}, first, min(last, n), sink, turn);
        at += last - first;
    }
}

// Workgroups before `prefix` walk the prefix, the others the sequences.
template <int kRW>
__global__ __launch_bounds__(Shape<kRW>::kThreads, 2) void mla_decode_q4_kernel(const MlaDecodeArgs A, int prefix) {
    __shared__ __attribute__((aligned(256))) Lds<kRW> lds;
    if (threadIdx.x < 2) lds.moved[threadIdx.x] = 0;
    __syncthreads();
    const int wg = blockIdx.x;
    if (wg < prefix) walk_prefix<kRW>(A, lds, wg);
    else walk_sequences<kRW>(A, lds, wg - prefix, int(gridDim.x) - prefix);
}

// Where the partial sums of a query row lie: `own` pieces of its sequence, then
// those of the prefix.  (false: it is already written)
struct Pieces {
    int own, n;
    int unit, lr, g0, stride;       // the sequence's: unit, row in it, first workgroup, rows a unit
    int pu, pr, pg0, pstride;       // the prefix's
    __device__ __forceinline__ bool find(const MlaDecodeArgs& A, int row) {
        const int unit_rows = A.tokens * A.heads;
        const int b = row / unit_rows, urow = row - b * unit_rows;   // row in the sequence
        stride = 32 * A.row_waves;
        const int blk = urow / stride;
        lr = urow - blk * stride;
        unit = b * A.row_blocks + blk;
        const int len = __builtin_amdgcn_readfirstlane(clamp_len(A, b));
        own = 0;
        g0 = 0;
        if (len > 0) {
            g0 = __builtin_amdgcn_readfirstlane(A.meta[2 * unit]);
            if (g0 < 0) return false;
            own = __builtin_amdgcn_readfirstlane(A.meta[2 * unit + 1]) - g0 + 1;
        }
        n = own;
        pu = pr = pg0 = 0;
        pstride = 32 * A.prefix_waves;
        if (A.prefix_len) {
            const int tiles = tiles_of(A.prefix_len);
            pu = row / pstride;
            pr = row - pu * pstride;
            pg0 = pu * A.prefix_line / A.prefix_per;
            n += (pu * A.prefix_line + tiles - 1) / A.prefix_per - pg0 + 1;
        }
        return true;
    }
    // piece i's statistics and the sums of `row`
    __device__ __forceinline__ void at(const MlaDecodeArgs& A, int i, const float*& part, const float*& ml) const {
        const bool mine = i < own;
        const int slot = mine ? (i == 0 ? unit : A.batch * A.row_blocks + g0 + i)
                              : (i == own ? pu : A.prefix_units + pg0 + (i - own));
        const size_t x = size_t(slot) * (mine ? stride : pstride) + (mine ? lr : pr);
        ml = (mine ? A.part_ml : A.pre_ml) + 2 * x;
        part = (mine ? A.part : A.pre_part) + x * kMlaLatent;
    }
};

// The sums of some of a row's pieces, relative to the largest reference among them.
template <int kLane>   // channels a lane
struct Joined {
    typedef float vec __attribute__((ext_vector_type(kLane)));
    float top = -INFINITY, total = 0.f;
    vec sum = 0.f;
    // pieces first, first + step, .. below n; eight at a time, all loads before their use
    __device__ __forceinline__ void add(const MlaDecodeArgs& A, const Pieces& P, int first, int step, int ch) {
        constexpr int kN = 8;
        for (int i0 = first; i0 < P.n; i0 += kN * step) {
            f32x2 ml[kN];
            vec x[kN];
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const float *part, *m;
                P.at(A, min(i0 + e * step, P.n - 1), part, m);
                ml[e] = *reinterpret_cast<const f32x2*>(m);
                x[e] = *reinterpret_cast<const vec*>(part + ch);
            }
            float most = top;
#pragma unroll
            for (int e = 0; e < kN; ++e) most = fmaxf(most, ml[e][0]);
            const float f = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(top - most);
            top = most;
            total *= f;
            sum *= f;
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                if (i0 + e * step >= P.n) break;
                take(ml[e][0], ml[e][1], x[e]);
            }
        }
    }
    // (a piece whose scores are all NaN has the reference -inf like one without
    // keys, but NaN for its sums)
    __device__ __forceinline__ void take(float m, float l, vec x) {
        const float w = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
        total = fmaf(l, w, total);
        sum += x * w;
    }
    __device__ __forceinline__ void put(const MlaDecodeArgs& A, int row, int ch, bool first) const {
        const float inv = total == 0.f ? 0.f : 1.f / total;
        uint32_t out[kLane / 2];
#pragma unroll
        for (int k = 0; k < kLane / 2; ++k) out[k] = pack_bf16(sum[2 * k] * inv, sum[2 * k + 1] * inv);
        __builtin_memcpy(__builtin_assume_aligned(A.o + int64_t(row) * kMlaLatent + ch, 2 * kLane), out, sizeof(out));
        if (A.lse && first) A.lse[row] = total == 0.f ? -INFINITY : fmaf(top, kLn2, logf(total));
    }
};

// Joins the partial sums of a query row, a wave per row: 8192 rows of about three
// pieces 10 us.
__global__ __launch_bounds__(kJoinThreads) void mla_join_q4_kernel(const MlaDecodeArgs A) {
    const int l = threadIdx.x & 63;
    const int row = blockIdx.x * (kJoinThreads / 64) + wave_id();
    Pieces P;
    if (row >= A.batch * A.tokens * A.heads || !P.find(A, row)) return;
    Joined<8> J;
    J.add(A, P, 0, 1, 8 * l);
    J.put(A, row, 8 * l, l == 0);
}

// The same by several waves a row: kParts parts of kWidth lanes share out its pieces
// (there may be hundreds), kLane channels a lane.
template <int kLane, int kWidth, int kParts>
__global__ __launch_bounds__(kWidth * kParts) void mla_join_parts_q4_kernel(const MlaDecodeArgs A) {
    typedef typename Joined<kLane>::vec vec;
    constexpr int kSlices = kMlaLatent / (kLane * kWidth);
    __shared__ float ml[kParts][2];
    __shared__ vec sums[kParts][kWidth];
    const int l = threadIdx.x % kWidth, part = threadIdx.x / kWidth;
    const int row = blockIdx.x / kSlices, ch = blockIdx.x % kSlices * (kMlaLatent / kSlices) + kLane * l;
    Pieces P;
    if (!P.find(A, row)) return;   // (the same for all)
    Joined<kLane> J;
    J.add(A, P, part, kParts, ch);
    if (l == 0) {
        ml[part][0] = J.top;
        ml[part][1] = J.total;
    }
    sums[part][l] = J.sum;
    __syncthreads();
    if (part > 0) return;
    const int parts = min(kParts, P.n);
    for (int k = 1; k < parts; ++k) J.top = fmaxf(J.top, ml[k][0]);
    J.total = 0.f;
    J.sum = 0.f;
    for (int k = 0; k < parts; ++k) J.take(ml[k][0], ml[k][1], sums[k][l]);
    J.put(A, row, ch, ch == 0);
}

// `prefix`: workgroups for the prefix in front; sequences: those of the batch behind.
template <int kRW>
hipError_t launch(const MlaDecodeArgs& A, bool prefix, bool sequences, hipStream_t stream) {
    const int64_t tiles = int64_t(A.prefix_units) * A.prefix_line;
    const int groups = prefix ? int((tiles + A.prefix_per - 1) / A.prefix_per) : 0;
    mla_decode_q4_kernel<kRW><<<dim3(unsigned(groups + (sequences ? kQ4Workgroups / kRW : 0))),
                                dim3(Shape<kRW>::kThreads), 0, stream>>>(A, groups);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mla_decode_q4(const MlaDecodeArgs& A, hipStream_t stream) {
    auto go = [&](int waves, bool prefix, bool sequences) {
        return waves == 2 ? launch<2>(A, prefix, sequences, stream) : launch<1>(A, prefix, sequences, stream);
    };
    const bool together = A.prefix_len > 0 && A.prefix_waves == A.row_waves;
    if (A.prefix_len > 0 && !together)
        if (hipError_t e = go(A.prefix_waves, true, false); e != hipSuccess) return e;
    if (hipError_t e = go(A.row_waves, together, true); e != hipSuccess) return e;
    const int rows = A.batch * A.tokens * A.heads;
    if (rows <= kEightRows)
        mla_join_parts_q4_kernel<2, 32, 32><<<dim3(unsigned(rows * 8)), dim3(1024), 0, stream>>>(A);
    else if (rows <= kWideRows)
        mla_join_parts_q4_kernel<4, 32, 32><<<dim3(unsigned(rows * 4)), dim3(1024), 0, stream>>>(A);
    else if (rows <= kFourRows)
        mla_join_parts_q4_kernel<8, 64, 4><<<dim3(unsigned(rows)), dim3(256), 0, stream>>>(A);
    else
        mla_join_q4_kernel<<<dim3(unsigned((rows + 3) / 4)), dim3(kJoinThreads), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace rda
