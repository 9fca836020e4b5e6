// rda_mla_decode_q4.hip -- absorbed latent attention over a paged latent cache
// in 4 bits.
#include <type_traits>

#include "rda_mla_q4.h"

namespace rda {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTile = 32;                        // cached rows per tile
constexpr int kTileBytes = kTile * kQ4Row;       // 12800
constexpr int kWaveRows = kTile / kWaves;        // rows of a tile that a wave fetches
constexpr int kWaveBytes = kWaveRows * kQ4Row;
constexpr int kBuf = 4;                          // tiles in flight or in use
constexpr int kValRows = 16;                     // rows unpacked at a time
constexpr int kValChannels = kMlaLatent / kWaves;
constexpr int kBlocks = kValChannels / 32;       // blocks of 32 channels a wave sums
constexpr int kValRow = kValChannels * 2;        // bytes
constexpr int kValBytes = kValRows * kValRow;
constexpr int kPieceTiles = 6;

template <int kRW>
struct Lds {
    unsigned char tile[kBuf][kTileBytes];
    unsigned char val[kWaves][kValBytes];   // a wave's own: unpacked values of its channels
    u32x4 p[2][kRW][kTile / 16][64];        // probabilities: [32 query rows][16 cached rows][lane]
    float top[kWaves][16];
    float l[kWaves][16];
    float mu[kRW * 32];
    float factor[kRW * 32];
    int moved[3];
    int scan[2 * kWaves];
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

// Row r of unpacked values (256 bytes) keeps 16-byte granule j at j ^ val_swz(r):
// eight rows written at one granule, and the rows and granules that a
// transposing read touches at a time, fall on distinct banks.
__device__ __forceinline__ int val_swz(int r) {
    return (r >> 1 & 1) * 10 | (r & 1) << 2 | (r >> 2 & 1);
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
    uint32_t scale;    // scale bytes of hi and lo
};

__device__ __forceinline__ void load_query(Query& Q, const uint16_t* row, int t) {
    u32x4 x[4][4];   // [product][16 bytes]
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int h = 0; h < 4; ++h)
            x[m][h] = *reinterpret_cast<const u32x4*>(
                row + 256 * (h >> 1) + 32 * (4 * (t >> 1) + m) + 16 * (t & 1) + 8 * (h & 1));
#pragma unroll
    for (int m = 0; m < 2; ++m)
        Q.pe[m] = __builtin_bit_cast(
            bf16x8, *reinterpret_cast<const u32x4*>(row + kMlaLatent + 32 * m + 8 * t));
    u16x2 most = {};
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, x[m][h][i] & 0x7fff7fffu));
    const uint32_t e = umax_over_quarters(max(uint32_t(most[0]), uint32_t(most[1]))) >> 7;
    // the largest value lands in [128, 256) of hi's scale
    const uint32_t sh = max(int(e) - 7, 24), sl = sh - 5;
    Q.scale = e == 255 ? 0xffffu : sh | sl << 8;
    const float fh = q4_scale(sh), fl = q4_scale(sl);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int d = 0; d < 2; ++d) {   // four values a dword
                s16x2 hi = {}, lo = {};
                const uint32_t a = x[m][h][2 * d], b = x[m][h][2 * d + 1];
                hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(bf16x2, a), fh, false);
                hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(bf16x2, b), fh, true);
                const uint32_t hw = __builtin_bit_cast(uint32_t, hi);
                const f32x2 ra = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hw, fh, false);
                const f32x2 rb = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hw, fh, true);
                lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(
                    lo, __uint_as_float(a << 16) - ra[0], __uint_as_float(a & 0xffff0000u) - ra[1], fl, false);
                lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(
                    lo, __uint_as_float(b << 16) - rb[0], __uint_as_float(b & 0xffff0000u) - rb[1], fl, true);
                Q.hi[m][2 * h + d] = int(hw);
                Q.lo[m][2 * h + d] = __builtin_bit_cast(int, lo);
            }
}

// One piece: tiles [t0, t1) of a source for 32 kRW query rows.
template <int kRW, bool kCausal>
__device__ __forceinline__ void piece(const MlaDecodeArgs& A, Lds<kRW>& lds, const Source& src, int t0,
                                      int t1, const Sink& sink) {
    constexpr int kRowWaves = 2 * kRW, kKW = kWaves / kRowWaves;   // row waves, key waves
    constexpr int kTB = kTile / 16 / kKW;                          // blocks of 16 cached rows a wave scores
    const int w = wave_id(), l = threadIdx.x & 63;
    const int rw = w % kRowWaves, kw = w / kRowWaves;
    const int c16 = l & 15, t = l >> 4, c32 = l & 31, g = l >> 5;
    const int end = min(src.len, t1 * kTile);
    const int all_see = kCausal ? src.len - (A.tokens - 1) : src.len;
    const float c = A.scale * kLog2e;
    const uint32_t tiles = lds_addr(&lds.tile[0][0]);
    const uint32_t val = lds_addr(&lds.val[w][0]);

    // lane j: the page of this wave's rows of tile `pages_from` + j
    int pages, pages_from = t0;
    auto load_pages = [&]() {
        const int k = (pages_from + l) * kTile + kWaveRows * w;
        pages = src.len > 0 ? src.table[k < src.len ? k >> A.page_shift : 0] : 0;
        pages = min(max(pages, 0), A.num_pages - 1);
    };
    load_pages();
    auto issue = [&](int tile, int buf) {
        if (tile - pages_from == 64) {
            pages_from = tile;
            load_pages();
        }
        const int k = tile * kTile + kWaveRows * w;
        const int page = __builtin_amdgcn_readlane(pages, tile - pages_from);
        q4_fetch_rows(reinterpret_cast<const char*>(A.cache) + int64_t(page) * A.page_stride +
                          int64_t(k & ((1 << A.page_shift) - 1)) * kQ4Row,
                      end - k, tiles + buf * kTileBytes + w * kWaveBytes, l);
    };
#pragma unroll 1
    for (int d = 0; d < kBuf - 1; ++d) issue(t0 + d, d);

    Query q;
    float m = -INFINITY, mu = 0.f, lsum = 0.f;
    const int qrow = min(16 * rw + c16, sink.rows - 1);
    load_query(q, A.q + (sink.row0 + qrow) * kMlaRow, t);
    const int limit = kCausal ? src.len - (A.tokens - 1 - (sink.first_row + qrow) / A.heads) : src.len;
    f32x16 acc[kRW][kBlocks];
#pragma unroll
    for (int rb = 0; rb < kRW; ++rb)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[rb][b][i] = 0.f;

    // this lane's addresses, from a tile's start
    const uint32_t krow = (kw * kTB * 16 + c16) * kQ4Row;                // the row it scores
    const uint32_t drow = c16 * kQ4Row + kQ4ScaleAt / kWaves * w + 16 * t;   // its part of the row it unpacks
    const uint32_t dscale = c16 * kQ4Row + kQ4ScaleAt + 4 * w;
    const uint32_t vput = val + c16 * kValRow;
    const int vr = 8 * g + (c16 >> 2), vlow = 2 * (t & 1) + ((c16 >> 1) & 1);
    uint32_t vget[2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
        vget[n] = val + (vr + 4 * n) * kValRow + 16 * (vlow ^ val_swz(vr + 4 * n)) + 8 * (c16 & 1);
    const uint32_t pput = lds_addr(&lds.p[0][rw >> 1][kw * kTB][16 * (rw & 1) + c16 + 32 * (t >> 1)]) + 8 * (t & 1);
    const bool idle = 16 * rw >= sink.rows;

    wait_vm<(kBuf - 2) * kQ4Fetch>();
    raw_barrier();
    f32x4 s[kTB];
    // this wave's scores of the tile at `tile`
    auto scores = [&](uint32_t tile) {
#pragma unroll
        for (int tb = 0; tb < kTB; ++tb) {
            const uint32_t row = tile + krow + tb * 16 * kQ4Row;
            const int sc = int(lds_read4(row + kQ4ScaleAt + 4 * t));
            f32x4 hi = zero4(), lo = zero4();   // (two chains: each product waits for the one before)
            each<4>([&](auto mm) {
                constexpr int n = decltype(mm)::value;
                const u32x4 k4 = lds_read_u4(row + 64 * t + 16 * n);
                const i32x8 a = {int(k4[0]), int(k4[1]), int(k4[2]), int(k4[3]), 0, 0, 0, 0};
                hi = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, q.hi[n], hi, 4, 0, n, sc, 0, int(q.scale));
                lo = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, q.lo[n], lo, 4, 0, n, sc, 1, int(q.scale));
            });
            hi = mfma_bf16(lds_read16(row + kQ4PeAt + 16 * t), q.pe[0], hi);
            lo = mfma_bf16(lds_read16(row + kQ4PeAt + 64 + 16 * t), q.pe[1], lo);
            s[tb] = hi + lo;
        }
    };
    if (!idle) scores(tiles);
    const int n_tiles = t1 - t0;
    for (int i = 0; i < n_tiles; ++i) {
        const int k0 = (t0 + i) * kTile, buf = i % kBuf, flag = i % 3;
        const uint32_t tile = tiles + buf * kTileBytes;
        const uint32_t pbuf = (i & 1) * sizeof(lds.p[0]);
        // 16 rows of this wave's 128 channels: a lane unpacks a group of a row
        u32x4 codes[kTile / kValRows];
        float unit[kTile / kValRows];
#pragma unroll
        for (int ch = 0; ch < kTile / kValRows; ++ch) {
            const uint32_t at = tile + ch * kValRows * kQ4Row;
            const uint32_t sb = (lds_read4(at + dscale) >> (8 * t)) & 255;
            codes[ch] = lds_read_u4(at + drow);
            // NaN groups are left out here: they have made the scores of all who
            // see them NaN, and no others may meet them as 0 x NaN
            unit[ch] = q4_scale(sb == kQ4Bad ? 0 : sb);
        }
        auto unpack = [&](int ch) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                lds_write_u4(vput + 16 * ((4 * t + j) ^ val_swz(c16)), q4_eight(codes[ch][j], unit[ch]));
        };
        auto store_p = [&]() {
#pragma unroll
            for (int tb = 0; tb < kTB; ++tb) {
                f32x4 e;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    e[x] = __builtin_amdgcn_exp2f(fmaf(s[tb][x], c, -mu));
                    lsum += e[x];
                }
                lds_write_u2(pput + pbuf + tb * sizeof(lds.p[0][0][0]),
                             u32x2{pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3])});
            }
        };
        float top = -INFINITY, before = 0.f;
        if (!idle) {
            if (k0 + kTile > all_see) {
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (k0 + 16 * (kw * kTB + tb) + 4 * t + x >= limit) s[tb][x] = -INFINITY;
            }
#pragma unroll
            for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
                for (int x = 0; x < 4; ++x) top = fmaxf(top, s[tb][x]);
            top = max_over_quarters(top);
            before = lsum;
            // the reference moves only when a row outgrows it by 2^8: the
            // probabilities go out against the one that stands, and again where it moves
            store_p();
            if (__any((top - m) * c > 8.f || (m == -INFINITY && top > m)) && l == 0) lds.moved[flag] = 1;
        }
        if (threadIdx.x == 0) lds.moved[flag == 2 ? 0 : flag + 1] = 0;
        unpack(0);
        wait_vm<(kBuf - 3) * kQ4Fetch>();   // this wave's part of the next tile
        raw_barrier();
        const int moved = lds.moved[flag];
        // the tile before is read: its memory takes the next one
        issue(t0 + i + kBuf - 1, (i + kBuf - 1) % kBuf);
        if (__builtin_amdgcn_readfirstlane(moved)) {
            if constexpr (kKW > 1) {
                if (t == 0) lds.top[w][c16] = top;
                raw_barrier();
            }
            if (!idle) {
                float mn = fmaxf(m, top);
                if constexpr (kKW > 1) {
#pragma unroll
                    for (int k = 0; k < kKW; ++k) mn = fmaxf(mn, lds.top[k * kRowWaves + rw][c16]);
                }
                const float mun = mn == -INFINITY ? 0.f : mn * c;
                const float a = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mu - mun);
                m = mn;
                mu = mun;
                lsum = before * a;
                if (kw == 0 && t == 0) lds.factor[16 * rw + c16] = a;
                store_p();
            }
            raw_barrier();
#pragma unroll
            for (int rb = 0; rb < kRW; ++rb) {
                const float f = lds.factor[32 * rb + c32];
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int x = 0; x < 16; ++x) acc[rb][b][x] *= f;
            }
        }
        // the scores of the next tile (zeros behind the last) beside this one's sums
        const uint32_t next = tiles + (buf + 1 == kBuf ? 0 : buf + 1) * kTileBytes;
        if (!idle) scores(next);
#pragma unroll
        for (int ch = 0; ch < kTile / kValRows; ++ch) {
            if (ch > 0) unpack(ch);
            bf16x8 pr[kRW];
#pragma unroll
            for (int rb = 0; rb < kRW; ++rb) pr[rb] = __builtin_bit_cast(bf16x8, lds.p[i & 1][rb][ch][l]);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const u32x2 x = lds_read_tr8(vget[0] ^ (64 * b));
                const u32x2 y = lds_read_tr8(vget[1] ^ (64 * b));
                const bf16x8 v = __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
#pragma unroll
                for (int rb = 0; rb < kRW; ++rb)
                    acc[rb][b] = mfma32(v, pr[rb], acc[rb][b]);
            }
        }
    }
    wait_vm<0>();   // the tiles behind the last: nothing may land later
    lsum = sum_over_quarters(lsum);
    if (t == 0) {
        lds.l[w][c16] = lsum;
        if (kw == 0) lds.mu[16 * rw + c16] = m == -INFINITY ? -INFINITY : mu;
    }
    raw_barrier();
#pragma unroll
    for (int rb = 0; rb < kRW; ++rb) {
        float total = 0.f;
#pragma unroll
        for (int k = 0; k < kKW; ++k) total += lds.l[k * kRowWaves + 2 * rb + (c32 >> 4)][c16];
        const int lr = 32 * rb + c32;
        if (w == rb && g == 0 && lr < sink.rows) {
            const float x = lds.mu[lr];
            if (!sink.final) *reinterpret_cast<f32x2*>(sink.ml + 2 * lr) = f32x2{x, total};
            else if (A.lse) A.lse[sink.row0 + lr] = total == 0.f ? -INFINITY : fmaf(x, kLn2, logf(total));
        }
        const float inv = !sink.final ? 1.f : total == 0.f ? 0.f : 1.f / total;
        // 32 channels at a time by way of LDS, so that they leave row by row
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const f32x16& a = acc[rb][b];
                const f32x4 y = {a[4 * x] * inv, a[4 * x + 1] * inv, a[4 * x + 2] * inv, a[4 * x + 3] * inv};
                lds_write_u4(val + c32 * 128 + 16 * ((2 * x + g) ^ (c32 & 7)), __builtin_bit_cast(u32x4, y));
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int r = 8 * x + (l >> 3), row = 32 * rb + r;
                const f32x4 y = __builtin_bit_cast(
                    f32x4, lds_read_u4(val + r * 128 + 16 * ((l & 7) ^ (r & 7))));
                if (row >= sink.rows) continue;
                const int ch = kValChannels * w + 32 * b + 4 * (l & 7);
                if (sink.final)
                    *reinterpret_cast<u32x2*>(A.o + (sink.row0 + row) * kMlaLatent + ch) =
                        u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
                else
                    *reinterpret_cast<f32x4*>(sink.part + size_t(row) * kMlaLatent + ch) = y;
            }
        }
    }
    raw_barrier();   // the next piece writes what this one has read
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

template <int kRW>
__global__ __launch_bounds__(kThreads, 2) void mla_decode_q4_kernel(const MlaDecodeArgs A) {
    __shared__ __attribute__((aligned(256))) Lds<kRW> lds;
    const int l = threadIdx.x & 63, w = wave_id(), wg = blockIdx.x;

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
        for (int k = 0; k < kWaves; ++k) {
            if (k < w) before += lds.scan[k];
            total += lds.scan[k];
        }
        return __builtin_amdgcn_readfirstlane(total);
    };
    auto tiles_at = [&](int b) { return b < A.batch ? tiles_of(clamp_len(A, b)) : 0; };
    if (threadIdx.x < 3) lds.moved[threadIdx.x] = 0;
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
    const int share = (total + kQ4Workgroups - 1) / kQ4Workgroups;
    const int units = A.batch * A.row_blocks;
    int per = max(share, min(A.min_tiles, (total + units - 1) / units));
    bool apart = false;
    if (units <= kQ4Workgroups && A.batch <= kThreads && share < 1 << 20) {
        int most = n0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
        if (l == 0) lds.scan[kWaves + w] = most;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kWaves; ++k) most = max(most, lds.scan[kWaves + k]);
        most = __builtin_amdgcn_readfirstlane(most);
        int each = max(A.min_tiles, total / (kQ4Workgroups - units / 2) + 1);
        for (int tries = 0; tries < 2 && !apart && each <= max(share, A.min_tiles) + kPieceTiles; ++tries) {
            if (most <= each + 2) each = most;
            const int padded = (n0 + each - 1) / each * each;
            int before;
            const int sum = block_sum(padded, before);
            if (sum * A.row_blocks <= each * kQ4Workgroups) {
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

    const int unit_rows = A.tokens * A.heads;
    int at = begin;
    while (at < end) {
        const int b = unit / A.row_blocks, blk = unit - b * A.row_blocks;
        const int len = __builtin_amdgcn_readfirstlane(clamp_len(A, b));
        const int n = tiles_of(len);
        if (n == 0) {   // the joining kernel writes these rows
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
        if (first == 0 && threadIdx.x == 0) {
            A.meta[2 * unit] = sink.final ? -1 : wg;
            A.meta[2 * unit + 1] = (at + n - 1) / per;
        }
        piece<kRW, true>(A, lds, Source{A.table + int64_t(b) * A.table_width, len}, first, last, sink);
        if (apart) break;
        at += last - first;
        first = 0;
        ++unit;
    }
}

// The prefix: every block of 32 kRW query rows walks all prefix rows.
template <int kRW>
__global__ __launch_bounds__(kThreads, 2) void mla_prefix_q4_kernel(const MlaDecodeArgs A) {
    __shared__ __attribute__((aligned(256))) Lds<kRW> lds;
    const int wg = blockIdx.x;
    const int rows = A.batch * A.tokens * A.heads;
    const int n = tiles_of(A.prefix_len);
    const int total = A.prefix_units * n;
    int at = A.prefix_per * wg;
    const int end = min(at + A.prefix_per, total);
    if (threadIdx.x < 3) lds.moved[threadIdx.x] = 0;
    __syncthreads();
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
        piece<kRW, false>(A, lds, Source{A.prefix_table, A.prefix_len}, first, last, sink);
        at += last - first;
    }
}

// Joins the partial sums of a query row, a wave per row (eight channels a lane).
__global__ __launch_bounds__(kThreads) void mla_join_q4_kernel(const MlaDecodeArgs A) {
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
    if (len > 0) {
        g0 = __builtin_amdgcn_readfirstlane(A.meta[2 * unit]);
        if (g0 < 0) return;   // already written
        np = __builtin_amdgcn_readfirstlane(A.meta[2 * unit + 1]) - g0 + 1;
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
            // (a piece whose scores are all NaN has the maximum -inf like one
            // without keys, but NaN for its sums)
            const float w = ml[e][0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[e][0] - most);
            total = fmaf(ml[e][1], w, total);
            sum[0] += x[e][0] * w;
            sum[1] += x[e][1] * w;
        }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    u32x4 out;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        out[k] = pack_bf16(sum[k >> 1][2 * (k & 1)] * inv, sum[k >> 1][2 * (k & 1) + 1] * inv);
    *reinterpret_cast<u32x4*>(A.o + int64_t(row) * kMlaLatent + 8 * l) = out;
    if (A.lse && l == 0) A.lse[row] = total == 0.f ? -INFINITY : fmaf(top, kLn2, logf(total));
}

template <int kRW>
void launch_private(const MlaDecodeArgs& A, hipStream_t stream) {
    mla_decode_q4_kernel<kRW><<<dim3(kQ4Workgroups), dim3(kThreads), 0, stream>>>(A);
}

template <int kRW>
void launch_prefix(const MlaDecodeArgs& A, hipStream_t stream) {
    const int total = A.prefix_units * ((A.prefix_len + kTile - 1) / kTile);
    mla_prefix_q4_kernel<kRW><<<dim3(unsigned((total + A.prefix_per - 1) / A.prefix_per)),
                                dim3(kThreads), 0, stream>>>(A);
}

}  // namespace

hipError_t launch_mla_decode_q4(const MlaDecodeArgs& A, hipStream_t stream) {
    if (A.prefix_len) {
        if (A.prefix_waves == 2) launch_prefix<2>(A, stream);
        else launch_prefix<1>(A, stream);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (A.row_waves == 2) launch_private<2>(A, stream);
    else launch_private<1>(A, stream);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int rows = A.batch * A.tokens * A.heads;
    mla_join_q4_kernel<<<dim3(unsigned((rows + 3) / 4)), dim3(kThreads), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace rda
