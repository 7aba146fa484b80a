// Tiles of 128 rows in the 8-bit format, as they are and transposed: encode, transpose and the gated activation's
// backward pass are one persistent kernel over tiles with different inputs and values.
//
// A CTA of 256 threads holds a tile's values as fp32 in registers; thread t (warp w, lane l) holds four rows from
// 4 * rg, rg = 4 * w + l / 8, and the 2 * CP columns from 2 * CP * (l % 8).  With CP = 8 a row's block of 128
// columns is eight neighbouring lanes (three shuffles for its largest magnitude, one 16-byte store of codes per
// lane).  A column's block of 128 rows is two shuffles and a maximum over the warps in shared memory; only the
// exponent that the scale needs of it is passed on, two columns to a word.  Four rows make a word of a column's
// codes, which pass through shared memory: a column's 128 codes are 8 chunks of 16 bytes, the chunk XORed with
// the column's lane, so that a warp's stores fall into different banks.
//
// What bounds these kernels next to the bytes is the shared-memory pipe (shuffles, staging) and the issue of
// instructions, hence the large thread tiles and the two-wide arithmetic.  Encoding 22016 x 4096 both ways (360 MB,
// 53 us at the copy rate): 85 us with two rows per thread, full-width maxima and 18 instructions per value, 63 us
// with 11.4.  The transpose issues 14 per value at 63 % of the issue rate (8192 x 4096: 20 us, bytes 10).  The gate's
// backward pass issues 58 at 47 % (5003 x 5504: 87 us, bytes 37) and saturates nothing: of the 8.3 cycles from one of a
// warp's instructions to its next, with four warps to a scheduler, fixed latencies take 1.4, shared memory and the special
// functions 1.0, the other warps' turns 0.9, global loads 0.8, the arithmetic pipe 0.6 and barriers 0.4.
//
// The next tiles' inputs arrive by tiled copies (a ring of stages) while a tile is worked on: with one tile per CTA
// loaded into registers, its loads, arithmetic and stores took their times one after another (242 us for the
// gate's backward pass).  bf16 inputs that such copies cannot read (16-byte alignment) are copied by the threads, each
// what it needs, a tile ahead (22016 x 4096 one element off, both ways: 86 us; loaded element by element 143).
#pragma once

#include "q8_tma.cuh"

namespace zs {

constexpr int kTileRp = 4;       // rows per thread
constexpr int kTileLanes = 8;    // lanes per row
constexpr int kTileThreads = 32 * kTileLanes;

template <int CP>            // column pairs per thread: tiles have 128 rows and 16 * CP columns
struct TilePos {
    int cc, rg;              // column chunk (2 * CP columns), row group (four rows)
    int64_t r0, c0;          // the tile's first row and column
    int rows, cols;          // valid rows and columns of the tile, 1 .. 128
    __device__ __forceinline__ bool row_ok(int p) const { return rg * kTileRp + p < rows; }
    __device__ __forceinline__ int chunk() const {            // valid columns of this thread's
        const int n = cols - cc * 2 * CP;
        return n < 0 ? 0 : n > 2 * CP ? 2 * CP : n;
    }
};

// A tile's row and column among the tiles.  A CTA goes from tile to tile in steps of the grid without dividing (with
// three divisions per tile: transpose of 8192 x 4096 20.8 us instead of 19.9, 3001 x 2047 encoded 13.9 and 13.6;
// encoding 22016 x 4096 62.0 and 63.3).
struct TileAt {
    uint32_t r, c;
    __device__ __forceinline__ void next(const TileAt& step, uint32_t tiles_c) {
        r += step.r;
        c += step.c;
        if (c >= tiles_c) {
            c -= tiles_c;
            ++r;
        }
    }
};

template <int CP>
__device__ __forceinline__ TilePos<CP> tile_pos(const TileAt& at, int64_t rows, int64_t cols) {
    TilePos<CP> t;
    t.cc = threadIdx.x % kTileLanes;
    t.rg = threadIdx.x / kTileLanes;
    t.r0 = (int64_t)at.r * 128;
    t.c0 = (int64_t)at.c * (2 * CP * kTileLanes);
    t.rows = rows - t.r0 < 128 ? (int)(rows - t.r0) : 128;
    t.cols = cols - t.c0 < 2 * CP * kTileLanes ? (int)(cols - t.c0) : 2 * CP * kTileLanes;
    return t;
}

// ------------------------------------------------------------------ 16 values at any address

struct V16 {
    uint32_t w[8];
};

// The matrix that accesses must stay in: its first and past its last byte.
struct Span {
    const uint8_t *lo, *hi;
};
__device__ __forceinline__ Span span_of(const uint16_t* p, int64_t ld, int64_t rows, int64_t cols) {
    return {reinterpret_cast<const uint8_t*>(p), reinterpret_cast<const uint8_t*>(p + (rows - 1) * ld + cols)};
}

// The 32 bytes that begin `off` (even, < 16) bytes into x.
__device__ __forceinline__ V16 shifted(uint32_t (&x)[12], uint32_t off) {
    if (off & 8) {
#pragma unroll
        for (int i = 0; i < 10; ++i) x[i] = x[i + 2];
    }
    if (off & 4) {
#pragma unroll
        for (int i = 0; i < 9; ++i) x[i] = x[i + 1];
    }
    V16 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v.w[i] = __funnelshift_r(x[i], x[i + 1], (off & 2) * 8);
    return v;
}

// Copies `bytes` <= 16 from src to dst, both 16-byte aligned, and zeros up to 16.
__device__ __forceinline__ void async16(uint8_t* dst, const uint8_t* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(su32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void async_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
// All but the newest group have landed.
__device__ __forceinline__ void async_wait_older() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// 16 bf16 values at p, read ahead of their use: the aligned 16-byte chunks that cover the n valid ones are copied to 48
// bytes of shared memory of the thread's own (fetch16), and shifted into place when their turn comes, the others 0
// (take16).  The caller commits and waits.  Loaded into registers they are shifted, and so waited for, at once: the
// norm of 16384 x 2047 took 107 us forward and 108 backward, 88 and 75 this way.
__device__ __forceinline__ void fetch16(uint8_t* slot, const uint16_t* p, int64_t n, const Span& s) {
    const uint8_t* at = reinterpret_cast<const uint8_t*>((uintptr_t)p & ~(uintptr_t)15);
    const int end = n <= 0 ? 0 : (int)((uintptr_t)p & 15) + 2 * (n < 16 ? (int)n : 16);       // of the bytes wanted
#pragma unroll
    for (int i = 0; i < 3; ++i, at += 16) {
        if (16 * i >= end) break;
        if (at >= s.lo) {
            async16(slot + 16 * i, at, s.hi - at < 16 ? (int)(s.hi - at) : 16);
        } else {                                 // the matrix starts inside this chunk
            for (int k = 0; k < 16; k += 2)
                if (at + k >= s.lo && at + k < s.hi) *reinterpret_cast<uint16_t*>(slot + k) = *reinterpret_cast<const uint16_t*>(at + k);
        }
    }
}
__device__ __forceinline__ V16 take16(const uint8_t* slot, const uint16_t* p, int64_t n) {
    uint32_t x[12];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(slot)[i];
        x[4 * i] = q.x; x[4 * i + 1] = q.y; x[4 * i + 2] = q.z; x[4 * i + 3] = q.w;
    }
    V16 v = shifted(x, (uint32_t)((uintptr_t)p & 15));
    if (n < 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v.w[i] &= 2 * i + 1 < n ? ~0u : 2 * i < n ? 0xffffu : 0u;
    }
    return v;
}
constexpr int kSlot = 48;

// ------------------------------------------------------------------ tiles in registers

// n (0 .. 16) bytes of w at p, which is 16-byte aligned.
__device__ __forceinline__ void store_codes(uint8_t* p, const uint4& w, int n) {
    if (n == 16) {
        __stcs(reinterpret_cast<uint4*>(p), w);
        return;
    }
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) p[i] = (uint8_t)(x[i >> 2] >> ((i & 3) * 8));
}
__device__ __forceinline__ uint4 load_codes(const uint8_t* p, int n) {
    if (n == 16) return __ldcs(reinterpret_cast<const uint4*>(p));
    uint32_t x[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) x[i >> 2] |= (uint32_t)p[i] << ((i & 3) * 8);
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// The scale exponent of a magnitude as the upper 16 bits of a sum (q8_scale_byte's): its maximum over a block is
// the block's, so that two columns' share a word.
__device__ __forceinline__ uint32_t scale_keys(float a, float b) {
    return __byte_perm(__float_as_uint(a) + 0x1fffffu, __float_as_uint(b) + 0x1fffffu, 0x7632);
}
__device__ __forceinline__ uint32_t key_byte(uint32_t key) {            // key: one column's 16 bits
    const int b = (int)(key >> 7) - 8;
    return (uint32_t)(b < 0 ? 0 : b);
}

// A thread's part of a tile's values: rows p, column pairs.
template <int CP>
struct TileValues {
    static constexpr int RP = kTileRp;
    float2 v[RP][CP];

    // Largest magnitude of each row's values.  Infinities become NaN, which the encoding leaves out of the
    // scale (rare: the test is one comparison on the maximum that the encoding needs anyway).
    __device__ __forceinline__ void find_tops(float (&top)[RP]) {
#pragma unroll
        for (int p = 0; p < RP; ++p) {
            top[p] = 0.f;
#pragma unroll
            for (int j = 0; j < CP; ++j) top[p] = q8_top2(top[p], v[p][j]);
        }
        float most = top[0];
#pragma unroll
        for (int p = 1; p < RP; ++p) most = fmaxf(most, top[p]);
        if (isinf(most)) {
#pragma unroll
            for (int p = 0; p < RP; ++p) {
                top[p] = 0.f;
#pragma unroll
                for (int j = 0; j < CP; ++j) {
                    v[p][j] = make_float2(q8_no_inf(v[p][j].x), q8_no_inf(v[p][j].y));
                    top[p] = q8_top2(top[p], v[p][j]);
                }
            }
        }
    }
    // The tile as it is.
    __device__ __forceinline__ void store_rows(const TilePos<CP>& t, const float (&top)[RP], const Q8& q) const {
        static_assert(2 * CP * kTileLanes == 128, "a row of the tile is a block");
        const int n = t.chunk();
        const int64_t r0 = t.r0 + t.rg * RP;
        uint8_t* codes = q.codes + r0 * q.ld + t.c0 + t.cc * 2 * CP;
        uint8_t* scales = q.scales + r0 * q.lds + (t.c0 >> 7);
#pragma unroll
        for (int p = 0; p < RP; ++p) {
            float m = top[p];
#pragma unroll
            for (int k = 1; k < kTileLanes; k <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, k));
            const uint32_t byte = q8_scale_byte(m);
            const float inv = q8_inverse(byte);
            uint32_t w[CP / 2];
#pragma unroll
            for (int k = 0; k < CP / 2; ++k) {
                const float2 a = q8_mul2(v[p][2 * k], make_float2(inv, inv)), b = q8_mul2(v[p][2 * k + 1], make_float2(inv, inv));
                w[k] = q8_pack4(a.x, a.y, b.x, b.y);
            }
            if (t.row_ok(p)) {
                store_codes(codes, make_uint4(w[0], w[1], w[2], w[3]), n);
                if (t.cc == 0) *scales = (uint8_t)byte;
            }
            codes += q.ld;
            scales += q.lds;
        }
    }
    // Scale keys of the columns over this warp's rows, into sh[warp][column pair].  Without find_tops before it
    // (no rows stored), infinities are found and replaced here.
    __device__ __forceinline__ void column_keys(uint32_t (*sh)[CP * kTileLanes]) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        float2 top[CP];
        auto tops = [&] {
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                top[j] = make_float2(0.f, 0.f);
#pragma unroll
                for (int p = 0; p < RP; p += 2)
                    top[j] = make_float2(q8_top2(top[j].x, make_float2(v[p][j].x, v[p + 1][j].x)),
                                         q8_top2(top[j].y, make_float2(v[p][j].y, v[p + 1][j].y)));
                most = q8_top2(most, top[j]);
            }
            return most;
        };
        if (isinf(tops())) {
#pragma unroll
            for (int p = 0; p < RP; ++p)
#pragma unroll
                for (int j = 0; j < CP; ++j) v[p][j] = make_float2(q8_no_inf(v[p][j].x), q8_no_inf(v[p][j].y));
            tops();
        }
        uint32_t key[CP];
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            key[j] = scale_keys(top[j].x, top[j].y);
#pragma unroll
            for (int k = kTileLanes; k < 32; k <<= 1) key[j] = __vmaxu2(key[j], __shfl_xor_sync(~0u, key[j], k));
        }
        if (lane < kTileLanes) {
            uint4* to = reinterpret_cast<uint4*>(&sh[warp][lane * CP]);
#pragma unroll
            for (int k = 0; k < CP / 4; ++k) to[k] = make_uint4(key[4 * k], key[4 * k + 1], key[4 * k + 2], key[4 * k + 3]);
        }
    }
    // Codes of the columns into word (8 chunks of 16 bytes per column), with inv[column] = 2^-e.  The chunk is XORed
    // with the column chunk, so that a warp's words fall into different banks.
    __device__ __forceinline__ void stage_columns(const TilePos<CP>& t, const float* inv, uint32_t* word) const {
        uint32_t* to = word + t.cc * 2 * CP * 32 + (((t.rg >> 2) ^ t.cc) << 2) + (t.rg & 3);
#pragma unroll
        for (int k = 0; k < CP / 2; ++k) {
            const float4 e = *reinterpret_cast<const float4*>(inv + t.cc * 2 * CP + k * 4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 s = h ? make_float2(e.z, e.w) : make_float2(e.x, e.y);
                float2 a[RP];
#pragma unroll
                for (int p = 0; p < RP; ++p) a[p] = q8_mul2(v[p][k * 2 + h], s);
                to[(k * 4 + h * 2) * 32] = q8_pack4(a[0].x, a[1].x, a[2].x, a[3].x);
                to[(k * 4 + h * 2 + 1) * 32] = q8_pack4(a[0].y, a[1].y, a[2].y, a[3].y);
            }
        }
    }
};

// Two columns' scales: the keys' maximum over the warps, the scale bytes into q, 2^-e into inv.
template <int CP>
__device__ __forceinline__ void column_scales(const TilePos<CP>& t, int pair, const uint32_t (*keys)[CP * kTileLanes], const Q8& q, float* inv) {
    uint32_t m = keys[0][pair];
#pragma unroll
    for (int k = 1; k < kTileLanes; ++k) m = __vmaxu2(m, keys[k][pair]);
    const uint32_t lo = key_byte(m & 0xffffu), hi = key_byte(m >> 16);
    *reinterpret_cast<float2*>(inv + pair * 2) = make_float2(q8_inverse(lo), q8_inverse(hi));
    uint8_t* to = q.scales + (t.c0 + pair * 2) * q.lds + (t.r0 >> 7);
    if (pair * 2 < t.cols) to[0] = (uint8_t)lo;
    if (pair * 2 + 1 < t.cols) to[q.lds] = (uint8_t)hi;
}

// Staged columns to their rows of q.
template <int CP>
__device__ __forceinline__ void store_columns(const TilePos<CP>& t, const uint32_t* word, const Q8& q) {
    const uint4* vec = reinterpret_cast<const uint4*>(word);
    const int part = threadIdx.x & 7;
    int n = t.rows - part * 16;
    n = n < 0 ? 0 : n > 16 ? 16 : n;
    uint8_t* to = q.codes + (t.c0 + (threadIdx.x >> 3)) * q.ld + t.r0 + part * 16;
    const int64_t step = 4 * kTileLanes * q.ld;
#pragma unroll
    for (int i = 0; i < CP / 2; ++i, to += step) {
        const int c = (threadIdx.x >> 3) + i * 4 * kTileLanes;
        const uint4 w = vec[c * 8 + (part ^ (c / (2 * CP)))];
        if (c < t.cols) store_codes(to, w, n);
    }
}

// ------------------------------------------------------------------ the kernel over tiles

enum { kTileEncode = 0, kTileTurn = 1, kTileGate = 2 };

struct TileArgs {
    const uint16_t* x;       // bf16 input (kTileEncode; kTileGate: dh), ldx elements between rows
    int64_t ldx;
    Q8 a, b;                 // 8-bit inputs (kTileTurn: a; kTileGate: gate and up)
    Q8 rows_out[2];          // the values as they are: encode q; gate dgate, dup
    Q8 cols_out[3];          // transposed: encode and turn q_t; gate dgate_t, dup_t, h_t
    int64_t rows, cols, tiles_c, tiles;
    unsigned int* error;
    long long wait_limit;
};

// Not TMA: the thread's slot for row p, and where the row's values are.
__device__ __forceinline__ uint8_t* tile_slot(const uint8_t* stage, int p) {
    return const_cast<uint8_t*>(stage) + (p * kTileThreads + threadIdx.x) * kSlot;
}
template <int CP>
__device__ __forceinline__ const uint16_t* tile_x(const TileArgs& a, const TilePos<CP>& t, int p) {
    return a.x + (t.r0 + t.rg * kTileRp + p) * a.ldx + t.c0 + t.cc * 2 * CP;
}
// Row p of the thread's part of a tile: bf16 values as packed words, from the stage or (not TMA) the thread's slots;
// decoded 8-bit values of an 8-bit tile at `from`.
template <bool TMA, int CP>
__device__ __forceinline__ void tile_bf16(const TileArgs& a, const TilePos<CP>& t, const uint8_t* stage, int p, uint32_t (&x)[CP]) {
    if constexpr (TMA) {
        const uint4* from = reinterpret_cast<const uint4*>(stage + (t.rg * kTileRp + p) * 4 * CP * kTileLanes + t.cc * 4 * CP);
#pragma unroll
        for (int k = 0; k < CP / 4; ++k) {
            const uint4 w = from[k];
            x[4 * k] = w.x; x[4 * k + 1] = w.y; x[4 * k + 2] = w.z; x[4 * k + 3] = w.w;
        }
    } else {
        static_assert(CP == 8, "16 columns");
        const V16 v = take16(tile_slot(stage, p), tile_x(a, t, p), t.row_ok(p) ? t.chunk() : 0);
#pragma unroll
        for (int j = 0; j < CP; ++j) x[j] = v.w[j];
    }
}
template <int CP>
__device__ __forceinline__ void tile_codes(const TilePos<CP>& t, const uint8_t* from, int p, uint32_t byte, float2 (&v)[CP]) {
    uint32_t w[CP / 2];
    const uint8_t* at = from + (t.rg * kTileRp + p) * 2 * CP * kTileLanes + t.cc * 2 * CP;
    if constexpr (CP == 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(at);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(at);
        w[0] = x.x; w[1] = x.y;
    }
    const float e = q8_scale(byte);
#pragma unroll
    for (int j = 0; j < CP; ++j) v[j] = q8_mul2(q8_unpack2(w[j >> 1] >> ((j & 1) * 16)), make_float2(e, e));
}

template <int KIND, bool TMA>
struct TileShape {
    // Column pairs per thread and lanes per row.  The transpose needs no whole row blocks, so its tiles are half as wide
    // and four CTAs fit an SM.  The others do best with large threads: the gate's backward pass at 5003 x 5504
    // takes 85 us so and 108 with 16 lanes of half the columns.
    static constexpr int kPairs = KIND == kTileTurn ? 4 : 8;
    static constexpr int kCols = 2 * kPairs * kTileLanes;
    // The gate's three values per element are taken one after another, each computed from the tile in shared memory:
    // all three in registers at once leave room for one CTA per SM, which is no faster (81 us at 5003 x 5504), and
    // this way only what is wanted is computed.
    static constexpr int kPasses = KIND == kTileGate ? 3 : 1;
    static constexpr int kX = KIND == kTileTurn || !TMA ? 0 : 128 * 128 * 2;      // bytes of a stage's copies: bf16 tile
    static constexpr int kA = KIND == kTileEncode ? 0 : 128 * kCols;                // and 8-bit tiles
    static constexpr int kB = KIND == kTileGate ? 128 * 128 : 0;
    static constexpr int kLoads = kX + kA + kB;
    static constexpr int kBf16 = KIND == kTileTurn ? 0 : TMA ? kX : kTileThreads * kTileRp * kSlot;    // of the bf16 tile or the slots
    static constexpr int kStage = kBf16 + kA + kB;
    static constexpr int kStages = KIND == kTileGate || (KIND == kTileEncode && !TMA) ? 1 : 2;
    static constexpr int kKeys = kTileLanes * kPairs * kTileLanes * 4;
    static constexpr int kSmem = 128 + kStages * kStage + 128 * kCols + kKeys + 512 + 64;
    static constexpr int kPerSm = KIND == kTileTurn ? 4 : 2;
};

// The gated activation's backward values: 0 the gate's gradient, 1 up's, 2 the activation itself.
template <int WHICH, bool TMA, int CP>
__device__ __forceinline__ void gate_values(TileValues<CP>& v, const TileArgs& a, const TilePos<CP>& t, const uint8_t* stage,
                                            const uint32_t (&sa)[kTileRp], const uint32_t (&sb)[kTileRp]) {
    const uint8_t* codes = stage + TileShape<kTileGate, TMA>::kBf16;
    const float2 one = make_float2(1.f, 1.f);
#pragma unroll
    for (int p = 0; p < kTileRp; ++p) {
        uint32_t x[CP] = {};
        float2 g[CP], u[CP];
        if constexpr (WHICH < 2) tile_bf16<TMA>(a, t, stage, p, x);
        tile_codes(t, codes, p, sa[p], g);
        if constexpr (WHICH != 1) tile_codes(t, codes + 128 * 128, p, sb[p], u);
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            const float2 d = make_float2(bf16_lo(x[j]), bf16_hi(x[j])), sig = q8_sigmoid2(g[j]);
            if constexpr (WHICH == 0) {
                const float2 rest = q8_fma2(sig, make_float2(-1.f, -1.f), one);                  // 1 - sigmoid
                v.v[p][j] = q8_mul2(q8_mul2(d, u[j]), q8_mul2(sig, q8_fma2(g[j], rest, one)));
            } else if constexpr (WHICH == 1) {
                v.v[p][j] = q8_mul2(d, q8_mul2(g[j], sig));
            } else {
                v.v[p][j] = q8_mul2(q8_mul2(g[j], sig), u[j]);
            }
        }
    }
}

template <int KIND, bool TMA>
__global__ void __launch_bounds__(kTileThreads, (TileShape<KIND, TMA>::kPerSm))
    k_q8_tiles(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_a,
               const __grid_constant__ CUtensorMap map_b, const __grid_constant__ TileArgs a) {
    using S = TileShape<KIND, TMA>;
    constexpr int RP = kTileRp, CP = S::kPairs;
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((128 - (su32(raw) & 127)) & 127);
    uint32_t* word = reinterpret_cast<uint32_t*>(base + S::kStages * S::kStage);                // [columns * 32]
    uint32_t (*keys)[CP * kTileLanes] = reinterpret_cast<uint32_t (*)[CP * kTileLanes]>(word + S::kCols * 32);    // [warps][column pairs]
    float* inv = reinterpret_cast<float*>(keys + kTileLanes);                                       // [128]
    uint64_t* full = reinterpret_cast<uint64_t*>(inv + 128);
    const int lane_row = threadIdx.x / kTileLanes * RP;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) mbar_init(full + i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    dependent_launch_prologue();

    const uint32_t tiles_c = (uint32_t)a.tiles_c, tiles = (uint32_t)a.tiles, grid = gridDim.x;
    const TileAt step = {grid / tiles_c, grid % tiles_c};
    auto load_stage = [&](int s, const TileAt& tile) {                              // thread 0
        if constexpr (S::kLoads > 0) {
            const int r0 = (int)(tile.r * 128), c0 = (int)(tile.c * S::kCols);
            uint8_t* at = base + s * S::kStage;
            mbar_expect_tx(full + s, S::kLoads);
            if constexpr (S::kX > 0) tma_load(at, &map_x, c0, r0, full + s);
            if constexpr (S::kA > 0) tma_load(at + S::kBf16, &map_a, c0, r0, full + s);
            if constexpr (S::kB > 0) tma_load(at + S::kBf16 + S::kA, &map_b, c0, r0, full + s);
        }
    };
    // scale bytes of the thread's rows, a tile ahead of their use
    uint32_t sa[RP] = {}, sb[RP] = {};
    auto load_scales = [&](const TileAt& tile) {
        if constexpr (S::kA > 0) {
            const uint32_t blk = tile.c * S::kCols >> 7;
            const int64_t r = (int64_t)tile.r * 128 + lane_row;
            const uint8_t *pa = a.a.scales + r * a.a.lds + blk, *pb = a.b.scales + r * a.b.lds + blk;
#pragma unroll
            for (int p = 0; p < RP; ++p, pa += a.a.lds, pb += a.b.lds) {
                sa[p] = r + p < a.rows ? *pa : 0;
                if constexpr (S::kB > 0) sb[p] = r + p < a.rows ? *pb : 0;
            }
        }
    };
    // not TMA: the thread's bf16 values of a tile, under way while the tile before is worked on
    constexpr bool kSlots = KIND != kTileTurn && !TMA;
    const Span sx = span_of(a.x, a.ldx, a.rows, a.cols);
    auto fetch_x = [&](const TileAt& tile) {
        const TilePos<CP> t = tile_pos<CP>(tile, a.rows, a.cols);
#pragma unroll
        for (int p = 0; p < RP; ++p) fetch16(tile_slot(base, p), tile_x(a, t, p), t.row_ok(p) ? t.chunk() : 0, sx);
        async_commit();
    };
    // the tile at work (then the next), and the one whose copies are issued next
    TileAt now = {blockIdx.x / tiles_c, blockIdx.x % tiles_c}, ahead = now;
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) {
        if (threadIdx.x == 0 && blockIdx.x + i * (int64_t)grid < tiles) load_stage(i, ahead);
        ahead.next(step, tiles_c);
    }
    load_scales(now);
    if constexpr (kSlots) fetch_x(now);
    int s = 0;
    uint32_t parity = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += grid) {
        const TilePos<CP> t = tile_pos<CP>(now, a.rows, a.cols);
        bool late = false;
        if constexpr (kSlots) async_wait_all();
        if constexpr (S::kLoads > 0) late = !mbar_wait_or_look(full + s, parity, a.wait_limit);
        const uint8_t* at = base + s * S::kStage;
#pragma unroll 1
        for (int pass = 0; pass < S::kPasses; ++pass) {
            const bool rows_wanted = KIND != kTileTurn && pass < 2 && a.rows_out[pass & 1].codes;
            const bool cols_wanted = a.cols_out[pass].codes;
            TileValues<CP> v;
            float top[RP];
            if (KIND != kTileGate || rows_wanted || cols_wanted) {
                if constexpr (KIND == kTileGate) {
                    if (pass == 0) gate_values<0, TMA>(v, a, t, at, sa, sb);
                    else if (pass == 1) gate_values<1, TMA>(v, a, t, at, sa, sb);
                    else gate_values<2, TMA>(v, a, t, at, sa, sb);
                } else {
#pragma unroll
                    for (int p = 0; p < RP; ++p) {
                        if constexpr (KIND == kTileEncode) {
                            uint32_t x[CP];
                            tile_bf16<TMA>(a, t, at, p, x);
#pragma unroll
                            for (int j = 0; j < CP; ++j) v.v[p][j] = make_float2(bf16_lo(x[j]), bf16_hi(x[j]));
                        } else {
                            tile_codes(t, at, p, sa[p], v.v[p]);
                        }
                    }
                }
                if (rows_wanted) v.find_tops(top);
                if (cols_wanted) v.column_keys(keys);
            }
            const bool last = pass == S::kPasses - 1;
            if (last) {
                now.next(step, tiles_c);
                if (tile + grid < tiles) {
                    load_scales(now);
                    if constexpr (kSlots) fetch_x(now);
                }
            }
            // A wait that ran out ends the CTA, after the copies still on their way.
            if (__syncthreads_or(late)) {
                if (threadIdx.x == 0) {
                    atomicCAS(a.error, 0u, ZS_DEVERR_TILE_WAIT);
                    for (int i = 0; i < S::kStages; ++i)
                        if (tile + i * (int64_t)grid < tiles)
                            mbar_wait(full + (s + i) % S::kStages, s + i >= S::kStages ? parity ^ 1 : parity, kDrainLimit);
                }
                return;
            }
            if (last) {                          // every thread has read the stage: its next tile may come
                if (threadIdx.x == 0 && tile + S::kStages * (int64_t)grid < tiles) load_stage(s, ahead);
                ahead.next(step, tiles_c);
                if (++s == S::kStages) {
                    s = 0;
                    parity ^= 1;
                }
            }
            if (cols_wanted && threadIdx.x < CP * kTileLanes) column_scales(t, threadIdx.x, keys, a.cols_out[pass], inv);
            if constexpr (KIND != kTileTurn)
                if (rows_wanted) v.store_rows(t, top, a.rows_out[pass & 1]);
            __syncthreads();
            if (cols_wanted) v.stage_columns(t, inv, word);
            __syncthreads();
            if (cols_wanted) store_columns(t, word, a.cols_out[pass]);
        }
    }
}

// ------------------------------------------------------------------ host

template <int KIND, bool TMA>
cudaError_t launch_tiles(TileArgs& a, cudaStream_t st) {
    using S = TileShape<KIND, TMA>;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = ready_once(ready, (const void*)k_q8_tiles<KIND, TMA>, S::kSmem);
    if (e != cudaSuccess) return e;
    a.tiles_c = (a.cols + S::kCols - 1) / S::kCols;
    a.tiles = a.tiles_c * ((a.rows + 127) / 128);
    if (a.tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.wait_limit = wait_limit().load(std::memory_order_relaxed);
    e = error_word(&a.error);
    CUtensorMap mx{}, ma{}, mb{};
    if (e == cudaSuccess && S::kX > 0) e = make_map(&mx, a.x, true, a.rows, a.cols, a.ldx * 2, 128, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e == cudaSuccess && S::kA > 0) e = make_map(&ma, a.a.codes, false, a.rows, a.cols, a.a.ld, 128, S::kCols, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e == cudaSuccess && S::kB > 0) e = make_map(&mb, a.b.codes, false, a.rows, a.cols, a.b.ld, 128, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e != cudaSuccess) return e;
    const int64_t room = (int64_t)q8_host::sm_count() * S::kPerSm;
    return launch_kernel(k_q8_tiles<KIND, TMA>, dim3((unsigned)(a.tiles < room ? a.tiles : room)), dim3(kTileThreads), S::kSmem, st, mx,
                         ma, mb, a);
}

}  // namespace zs
