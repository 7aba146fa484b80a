// A 128 x 128 tile of fp32 values in the registers of one CTA, and its 8-bit forms along both directions.
//
// 256 threads; thread t (warp w, lane l) holds rows 4 * rg .. + 3 with rg = 4 * w + l / 8 and the 16
// columns 16 * (l % 8) ..: v[p][j] is row 4 * rg + p, column 16 * (l % 8) + j.  A row's block of 128
// columns is then eight neighbouring lanes (three shuffles for its largest magnitude, one 16-byte store
// of codes per lane); a column's block of 128 rows is two shuffles and a maximum over the eight warps in
// shared memory.  Four rows per thread make one 32-bit word of a column's codes, so the transpose
// through shared memory is 16 word stores and 4 16-byte loads per thread; the word index is XORed with
// the column chunk, which puts a warp's 32 words into 32 banks.
#pragma once

#include "q8.cuh"

namespace zs {

constexpr int kTileThreads = 256;

struct TilePos {
    int cc, rg;              // column chunk (16 columns), row group (4 rows)
    int64_t r0, c0;          // the tile's first row and column
    int rows, cols;          // valid rows and columns of the tile, 1 .. 128
    __device__ __forceinline__ bool row_ok(int p) const { return rg * 4 + p < rows; }
    __device__ __forceinline__ int chunk() const {            // valid columns of this thread's 16
        const int n = cols - cc * 16;
        return n < 0 ? 0 : n > 16 ? 16 : n;
    }
};

__device__ __forceinline__ TilePos tile_pos(int64_t tile, int64_t tiles_c, int64_t rows, int64_t cols) {
    TilePos t;
    t.cc = threadIdx.x & 7;
    t.rg = threadIdx.x >> 3;
    const int64_t tr = tile / tiles_c;
    t.r0 = tr * 128;
    t.c0 = (tile - tr * tiles_c) * 128;
    t.rows = rows - t.r0 < 128 ? (int)(rows - t.r0) : 128;
    t.cols = cols - t.c0 < 128 ? (int)(cols - t.c0) : 128;
    return t;
}

// n (0 .. 16) bytes of w at p, which is 16-byte aligned.
__device__ __forceinline__ void store_codes(uint8_t* p, const uint4& w, int n) {
    if (n == 16) {
        *reinterpret_cast<uint4*>(p) = w;
        return;
    }
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    for (int i = 0; i < n; ++i) p[i] = (uint8_t)(x[i >> 2] >> ((i & 3) * 8));
}
__device__ __forceinline__ uint4 load_codes(const uint8_t* p, int n) {
    if (n == 16) return __ldcs(reinterpret_cast<const uint4*>(p));
    uint32_t x[4] = {0, 0, 0, 0};
    for (int i = 0; i < n; ++i) x[i >> 2] |= (uint32_t)p[i] << ((i & 3) * 8);
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// 16 bf16 values at p (n of them valid, the others 0) as packed words.
template <bool WIDE>
__device__ __forceinline__ void load_bf16_16(const uint16_t* p, int n, uint32_t (&w)[8]) {
    if (WIDE && n == 16) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p)), b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
            w[i] = lo | (hi << 16);
        }
    }
}

// Replaces infinities by NaN in this thread's values when there are any (rare: the test is one
// comparison on the maximum that the encoding needs anyway); `top` then leaves them out.
__device__ __forceinline__ void tile_row_tops(float (&v)[4][16], float (&top)[4]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        top[p] = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) top[p] = q8_top(top[p], v[p][j]);
    }
    if (isinf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])))) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            top[p] = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                v[p][j] = q8_no_inf(v[p][j]);
                top[p] = q8_top(top[p], v[p][j]);
            }
        }
    }
}

// Writes the tile as it is: `top` from tile_row_tops.
__device__ __forceinline__ void tile_store_rows(const TilePos& t, const float (&v)[4][16], const float (&top)[4],
                                                const Q8& q) {
    const int n = t.chunk();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        float m = top[p];
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 4));
        const uint32_t byte = q8_scale_byte(m);
        const float inv = q8_inverse(byte);
        uint4 w;
        w.x = q8_pack4(v[p][0] * inv, v[p][1] * inv, v[p][2] * inv, v[p][3] * inv);
        w.y = q8_pack4(v[p][4] * inv, v[p][5] * inv, v[p][6] * inv, v[p][7] * inv);
        w.z = q8_pack4(v[p][8] * inv, v[p][9] * inv, v[p][10] * inv, v[p][11] * inv);
        w.w = q8_pack4(v[p][12] * inv, v[p][13] * inv, v[p][14] * inv, v[p][15] * inv);
        if (t.row_ok(p)) {
            const int64_t r = t.r0 + t.rg * 4 + p;
            store_codes(q.codes + r * q.ld + t.c0 + t.cc * 16, w, n);
            if (t.cc == 0) q.scales[r * q.lds + (t.c0 >> 7)] = (uint8_t)byte;
        }
    }
}

struct TileShared {
    float top[8][128];       // largest magnitude of a column in a warp's 16 rows
    float inv[128];          // 2^-e of a column's block
    uint32_t word[128 * 32]; // a column's codes, 32 words each, word index ^ (chunk * 4)
};

// Writes the transposed tile: column c of the tile is row c0 + c of q.  Infinities are gone already
// (tile_row_tops).  Every thread of the CTA calls it; `sh` may be reused at once by the next call.
__device__ __forceinline__ void tile_store_columns(const TilePos& t, const float (&v)[4][16], const Q8& q,
                                                   TileShared& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float m = q8_top(q8_top(q8_top(q8_top(0.f, v[0][j]), v[1][j]), v[2][j]), v[3][j]);
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 8));
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 16));
        if (lane < 8) sh.top[warp][t.cc * 16 + j] = m;
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        const int c = threadIdx.x;
        float m = sh.top[0][c];
#pragma unroll
        for (int k = 1; k < 8; ++k) m = fmaxf(m, sh.top[k][c]);
        const uint32_t byte = q8_scale_byte(m);
        sh.inv[c] = q8_inverse(byte);
        if (c < t.cols) q.scales[(t.c0 + c) * q.lds + (t.r0 >> 7)] = (uint8_t)byte;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int c = t.cc * 16 + j;
        const float inv = sh.inv[c];
        sh.word[c * 32 + (t.rg ^ (t.cc << 2))] = q8_pack4(v[0][j] * inv, v[1][j] * inv, v[2][j] * inv, v[3][j] * inv);
    }
    __syncthreads();
    const uint4* vec = reinterpret_cast<const uint4*>(sh.word);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = threadIdx.x + i * kTileThreads, c = k >> 3, part = k & 7;
        const uint4 w = vec[c * 8 + (part ^ (c >> 4))];
        int n = t.rows - part * 16;
        n = n < 0 ? 0 : n > 16 ? 16 : n;
        if (c < t.cols) store_codes(q.codes + (t.c0 + c) * q.ld + t.r0 + part * 16, w, n);
    }
}

}  // namespace zs
