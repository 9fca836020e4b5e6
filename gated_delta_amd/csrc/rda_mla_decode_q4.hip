// rda_mla_decode_q4.hip -- absorbed latent attention over a paged latent cache
// in 4 bits.
#include <type_traits>

#include "rda_mla_q4.h"

namespace rda {
namespace {

typedef const __attribute__((address_space(4))) int32_t const_i32;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kTile = 64;                        // cached rows per tile
constexpr int kTileBytes = kTile * kQ4Row;       // 25600
constexpr int kWaveRows = 16;                    // rows of a tile that a wave fetches
constexpr int kWaveBytes = kWaveRows * kQ4Row;   // 6400
constexpr int kDma = 7;                          // transfers for them: 400 granules of 16 bytes
constexpr int kValRows = 32;                     // rows unpacked at a time
constexpr int kValBytes = kValRows * 256;        // of 128 channels
constexpr int kPieceTiles = 3;

__device__ const __attribute__((aligned(16))) uint32_t kZeros[4] = {};

template <int kRW>
struct Lds {
    static constexpr int kBuf = kRW == 4 ? 3 : 4;   // tiles in flight or in use
    unsigned char tile[kBuf][kTileBytes];
    unsigned char val[4][kValBytes];     // a wave's own: unpacked values, 128 channels
    u32x4 p[2][kRW][4][64];              // probabilities: [row block][16 cached rows][lane]
    float top[4][32];
    float l[4][32];
    float mu[kRW * 32];
    float factor[kRW * 32];
    int moved[3];
    int scan[8];
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
__device__ __forceinline__ void lds_write_u4(uint32_t a, u32x4 x) {
    *(lds_u32x4*)(lds_char*)uintptr_t(a) = x;
}

// Row r of unpacked values keeps 16-byte granule j at j ^ val_swz(r): sixteen
// rows written at one granule, and the rows and granules that a transposing
// read touches at a time, fall on distinct banks.
__device__ __forceinline__ int val_swz(int r) { return (r & 3) << 2 | (r >> 3 & 1) << 1 | (r >> 2 & 1); }

__device__ __forceinline__ int clamp_len(const MlaDecodeArgs& A, int b) {
    const int64_t most = int64_t(A.table_width) << A.page_shift;
    const int n = A.kv_lens[b];
    return A.num_pages > 0 && n > 0 ? int(n < most ? n : most) : 0;
}

struct Source {
    const int32_t* table;
    int len;
};

__device__ __forceinline__ int page_of(const MlaDecodeArgs& A, const Source& src, int k) {
    const int at = k < src.len ? k >> A.page_shift : 0;
    return src.len > 0 ? min(max(((const_i32*)src.table)[at], 0), A.num_pages - 1) : 0;
}

// Sixteen rows [k, k + 16) into LDS as they lie, one behind the other: two
// groups of eight (a page holds whole groups of eight).  Rows from `end` on are
// read as zeros.
__device__ __forceinline__ void fetch_rows(const MlaDecodeArgs& A, const int (&page)[2], int k, int end,
                                           uint32_t lds, int lane) {
    const char* base[2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
        base[n] = reinterpret_cast<const char*>(A.cache) + int64_t(page[n]) * A.page_stride +
                  int64_t((k + 8 * n) & ((1 << A.page_shift) - 1)) * kQ4Row;
    const int l = here(lane);
    const int valid = end - k;
    if (valid >= kWaveRows) {
#pragma unroll
        for (int i = 0; i < 3; ++i) dma16_at(base[0], 16 * l + 1024 * i, lds + 1024 * i);
        dma16_from(l < 8 ? base[0] + 16 * l + 1024 * 3 : base[1] + 16 * l - 128, lds + 1024 * 3);
#pragma unroll
        for (int i = 4; i < 6; ++i) dma16_at(base[1], 16 * l + 1024 * i - 3200, lds + 1024 * i);
        if (l < 16) dma16_at(base[1], 16 * l + 1024 * 6 - 3200, lds + 1024 * 6);
    } else {
#pragma unroll
        for (int i = 0; i < kDma; ++i) {
            const int g = 64 * i + l, row = g * 5243 >> 17;   // g / 25
            const char* from = g < 200 ? base[0] + 16 * g : base[1] + 16 * (g - 200);
            if (row >= valid) from = reinterpret_cast<const char*>(kZeros);
            if (i < kDma - 1 || l < 16) dma16_from(from, lds + 1024 * i);
        }
    }
}

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
    constexpr int kKW = 4 / kRW, kTB = kRW;
    constexpr int kBuf = Lds<kRW>::kBuf;
    const int w = wave_id(), l = threadIdx.x & 63;
    const int rw = w % kRW, kw = w / kRW;
    const int c16 = l & 15, t = l >> 4, c32 = l & 31, g = l >> 5;
    const int end = min(src.len, t1 * kTile);
    const int all_see = kCausal ? src.len - (A.tokens - 1) : src.len;
    const float c = A.scale * kLog2e;
    const uint32_t tiles = lds_addr(&lds.tile[0][0]);
    const uint32_t val = lds_addr(&lds.val[w][0]);

    int page[2];
    auto pages = [&](int tile) {
#pragma unroll
        for (int n = 0; n < 2; ++n) page[n] = page_of(A, src, tile * kTile + kWaveRows * w + 8 * n);
    };
    auto issue = [&](int tile, int buf) {
        fetch_rows(A, page, tile * kTile + kWaveRows * w, end, tiles + buf * kTileBytes + w * kWaveBytes, l);
        pages(tile + 1);
    };
    pages(t0);
#pragma unroll 1
    for (int d = 0; d < kBuf - 1; ++d) issue(t0 + d, d);

    Query q[2];
    int limit[2];
    float m[2] = {-INFINITY, -INFINITY}, mu[2] = {0.f, 0.f}, lsum[2] = {0.f, 0.f};
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) {
        const int row = min(32 * rw + 16 * nb + c16, sink.rows - 1);
        load_query(q[nb], A.q + (sink.row0 + row) * kMlaRow, t);
        limit[nb] = kCausal ? src.len - (A.tokens - 1 - (sink.first_row + row) / A.heads) : src.len;
    }
    f32x16 acc[kRW][4];
#pragma unroll
    for (int rb = 0; rb < kRW; ++rb)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[rb][b][i] = 0.f;

    // this lane's addresses, from a tile's start
    const uint32_t krow = (kw * kTB * 16 + c16) * kQ4Row;            // its row's scores
    const uint32_t drow = c32 * kQ4Row;                              // the row it unpacks
    const int vr = 8 * g + (c16 >> 2), vlow = 2 * (t & 1) + ((c16 >> 1) & 1);
    uint32_t va[2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
        va[n] = val + (vr + 4 * n) * 256 + 16 * (vlow ^ val_swz(vr + 4 * n)) + 8 * (c16 & 1);
    const bool idle = 32 * rw >= sink.rows;
    const int row_blocks = min(kRW, (sink.rows + 31) / 32);

    if constexpr (kKW == 1 || kRW == 2) {
        wait_vm<(kBuf - 2) * kDma>();
        raw_barrier();
    }
    const int n_tiles = t1 - t0;
    for (int i = 0; i < n_tiles; ++i) {
        const int k0 = (t0 + i) * kTile, buf = i % kBuf, flag = i % 3;
        const uint32_t tile = tiles + buf * kTileBytes;
        if constexpr (kRW == 1) wait_vm<(kBuf - 2) * kDma>();   // its own 16 rows have landed
        f32x4 s[kTB][2];
        float p[2][2];   // (reference moves)
        (void)p;
        auto store_p = [&]() {
#pragma unroll
            for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
                    f32x4 e;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        e[x] = __builtin_amdgcn_exp2f(fmaf(s[tb][nb][x], c, -mu[nb]));
                        lsum[nb] += e[x];
                    }
                    const u32x2 y = {pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3])};
                    *reinterpret_cast<u32x2*>(
                        reinterpret_cast<char*>(&lds.p[i & 1][rw][kw * kTB + tb][16 * nb + c16 + 32 * (t >> 1)]) +
                        8 * (t & 1)) = y;
                }
        };
        float top[2], before[2];
        if (!idle) {
#pragma unroll
            for (int tb = 0; tb < kTB; ++tb) {
                const uint32_t row = tile + krow + tb * 16 * kQ4Row;
                const int sc = int(lds_read4(row + kQ4ScaleAt + 4 * t));
                s[tb][0] = s[tb][1] = zero4();
                each<4>([&](auto mm) {
                    constexpr int n = decltype(mm)::value;
                    const u32x4 k4 = lds_read_u4(row + 64 * t + 16 * n);
                    i32x8 a = {int(k4[0]), int(k4[1]), int(k4[2]), int(k4[3]), 0, 0, 0, 0};
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) {
                        s[tb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            a, q[nb].hi[n], s[tb][nb], 4, 0, n, sc, 0, int(q[nb].scale));
                        s[tb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            a, q[nb].lo[n], s[tb][nb], 4, 0, n, sc, 1, int(q[nb].scale));
                    }
                });
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const bf16x8 pe = lds_read16(row + kQ4PeAt + 64 * n + 16 * t);
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) s[tb][nb] = mfma_bf16(pe, q[nb].pe[n], s[tb][nb]);
                }
            }
            if (k0 + kTile > all_see) {
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (k0 + 16 * (kw * kTB + tb) + 4 * t + x >= limit[nb]) s[tb][nb][x] = -INFINITY;
            }
            bool move = false;
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
                float y = s[0][nb][0];
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
                    for (int x = 0; x < 4; ++x) y = fmaxf(y, s[tb][nb][x]);
                top[nb] = max_over_quarters(y);
                move |= (top[nb] - m[nb]) * c > 8.f || (m[nb] == -INFINITY && top[nb] > m[nb]);
                before[nb] = lsum[nb];
            }
            // the reference moves only when a row outgrows it by 2^8: the
            // probabilities go out against the one that stands, and again where it moves
            store_p();
            if (__any(move) && l == 0) lds.moved[flag] = 1;
        }
        if (threadIdx.x == 0) lds.moved[flag == 2 ? 0 : flag + 1] = 0;
        if constexpr (kRW > 1) wait_vm<(kBuf - 3) * kDma>();   // this wave's part of the next tile
        raw_barrier();
        if (__builtin_amdgcn_readfirstlane(lds.moved[flag])) {
            if constexpr (kKW > 1) {
                if (t == 0) {
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) lds.top[w][16 * nb + c16] = top[nb];
                }
                raw_barrier();
            }
            if (!idle) {
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
                    float mn = fmaxf(m[nb], top[nb]);
                    if constexpr (kKW > 1) {
#pragma unroll
                        for (int k = 0; k < kKW; ++k) mn = fmaxf(mn, lds.top[k * kRW + rw][16 * nb + c16]);
                    }
                    const float mun = mn == -INFINITY ? 0.f : mn * c;
                    const float a = m[nb] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mu[nb] - mun);
                    m[nb] = mn;
                    mu[nb] = mun;
                    lsum[nb] = before[nb] * a;
                    if (kw == 0 && t == 0) lds.factor[32 * rw + 16 * nb + c16] = a;
                }
                store_p();
            }
            raw_barrier();
#pragma unroll
            for (int rb = 0; rb < kRW; ++rb) {
                const float f = lds.factor[32 * rb + c32];
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int x = 0; x < 16; ++x) acc[rb][b][x] *= f;
            }
        }
        // the tile before is read: its memory takes the next one
        issue(t0 + i + kBuf - 1, (i + kBuf - 1) % kBuf);
#pragma unroll
        for (int ch = 0; ch < kTile / kValRows; ++ch) {
            // this wave's 128 channels of 32 rows as bf16
            const uint32_t row = tile + drow + ch * kValRows * kQ4Row;
            const uint32_t sc = lds_read4(row + kQ4ScaleAt + 4 * w);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const u32x4 x = lds_read_u4(row + 64 * w + 32 * n + 16 * g);
                const uint32_t sb = (sc >> (16 * n + 8 * g)) & 255;
                // NaN groups are left out here: they have made the scores of all
                // who see them NaN, and no others may meet them as 0 x NaN
                const float f = q4_scale(sb == kQ4Bad ? 0 : sb);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    lds_write_u4(val + c32 * 256 + 16 * ((4 * (2 * n + g) + j) ^ val_swz(c32)), q4_eight(x[j], f));
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bf16x8 pr[kRW];
#pragma unroll
                for (int rb = 0; rb < kRW; ++rb)
                    pr[rb] = __builtin_bit_cast(bf16x8, lds.p[i & 1][rb][2 * ch + kk][l]);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const u32x2 x = lds_read_tr8((va[0] ^ (64 * b)) + kk * 16 * 256);
                    const u32x2 y = lds_read_tr8((va[1] ^ (64 * b)) + kk * 16 * 256);
                    const bf16x8 v = __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
#pragma unroll
                    for (int rb = 0; rb < kRW; ++rb)
                        acc[rb][b] = mfma32(v, pr[rb], acc[rb][b]);
                }
            }
        }
    }
    (void)row_blocks;
    wait_vm<0>();   // the tiles behind the last: nothing may land later
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) {
        const float y = sum_over_quarters(lsum[nb]);
        if (t == 0) {
            lds.l[w][16 * nb + c16] = y;
            if (kw == 0) lds.mu[32 * rw + 16 * nb + c16] = m[nb] == -INFINITY ? -INFINITY : mu[nb];
        }
    }
    raw_barrier();
#pragma unroll
    for (int rb = 0; rb < kRW; ++rb) {
        float total = 0.f;
#pragma unroll
        for (int k = 0; k < kKW; ++k) total += lds.l[k * kRW + rb][c32];
        const int lr = 32 * rb + c32;
        if (w == rb % 4 && g == 0 && lr < sink.rows) {
            const float x = lds.mu[lr];
            if (!sink.final) *reinterpret_cast<f32x2*>(sink.ml + 2 * lr) = f32x2{x, total};
            else if (A.lse) A.lse[sink.row0 + lr] = total == 0.f ? -INFINITY : fmaf(x, kLn2, logf(total));
        }
        const float inv = !sink.final ? 1.f : total == 0.f ? 0.f : 1.f / total;
        // 64 channels at a time by way of LDS, so that they leave row by row
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const f32x16& a = acc[rb][2 * h + b];
                    const f32x4 y = {a[4 * x] * inv, a[4 * x + 1] * inv, a[4 * x + 2] * inv, a[4 * x + 3] * inv};
                    lds_write_u4(val + c32 * 256 + 16 * ((8 * b + 2 * x + g) ^ c16), __builtin_bit_cast(u32x4, y));
                }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int r = 4 * x + t, row = 32 * rb + r;
                const f32x4 y = __builtin_bit_cast(f32x4, lds_read_u4(val + r * 256 + 16 * (c16 ^ (r & 15))));
                if (row >= sink.rows) continue;
                const int ch = 128 * w + 64 * h + 4 * c16;
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
__global__ __launch_bounds__(kThreads, 1) void mla_decode_q4_kernel(const MlaDecodeArgs A) {
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
        for (int k = 0; k < 4; ++k) {
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
    const int share = (total + kMlaWorkgroups - 1) / kMlaWorkgroups;
    const int units = A.batch * A.row_blocks;
    int per = max(share, min(A.min_tiles, (total + units - 1) / units));
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
            if (most <= each + 1) each = most;
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
__global__ __launch_bounds__(kThreads, 1) void mla_prefix_q4_kernel(const MlaDecodeArgs A) {
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
    mla_decode_q4_kernel<kRW><<<dim3(kMlaWorkgroups), dim3(kThreads), 0, stream>>>(A);
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
        if (A.prefix_waves == 4) launch_prefix<4>(A, stream);
        else launch_prefix<1>(A, stream);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (A.row_waves == 4) launch_private<4>(A, stream);
    else if (A.row_waves == 2) launch_private<2>(A, stream);
    else launch_private<1>(A, stream);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int rows = A.batch * A.tokens * A.heads;
    mla_join_q4_kernel<<<dim3(unsigned((rows + 3) / 4)), dim3(kThreads), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace rda
