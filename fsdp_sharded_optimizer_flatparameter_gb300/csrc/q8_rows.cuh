// Rows of bf16 matrices and of the 8-bit format, 16 neighbouring columns per thread.
#pragma once

#include "q8_tile.cuh"

namespace zs {

// ------------------------------------------------------------------ vectors of 16 columns
//
// A thread holds 16 neighbouring columns (32 bytes of bf16, 16 codes), so eight neighbouring lanes hold a
// block of the format.  Aligned rows move 32 bytes per access.  Rows at other addresses (an odd width, a
// view into a flat buffer) are read as the aligned 16-byte chunks that cover a thread's columns, shifted
// into place, and written as the aligned chunks that a thread and its right neighbour make up together;
// element by element a row of 2047 columns took 16 accesses per thread, each touching 32 sectors.  Where rows are
// read ahead, the chunks go through shared memory (fetch16, take16).

// 16 bf16 values at p, n of them valid (n may be <= 0 or > 16), the others 0.
template <bool WIDE>
__device__ __forceinline__ V16 load16(const uint16_t* p, int64_t n, const Span& s) {
    V16 v;
    if (WIDE) {
        if (n >= 16) {
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                           "=r"(v.w[7])
                         : "l"(p));
            return v;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
            v.w[i] = lo | (hi << 16);
        }
        return v;
    }
    const uint8_t* at = reinterpret_cast<const uint8_t*>((uintptr_t)p & ~(uintptr_t)15);
    const uint32_t off = (uint32_t)((uintptr_t)p & 15);
    uint32_t x[12];
    if (n >= 16 && at >= s.lo && at + 48 <= s.hi) {
        const uint4* q = reinterpret_cast<const uint4*>(at);
        const uint4 q0 = q[0], q1 = q[1], q2 = q[2];
        x[0] = q0.x; x[1] = q0.y; x[2] = q0.z; x[3] = q0.w;
        x[4] = q1.x; x[5] = q1.y; x[6] = q1.z; x[7] = q1.w;
        x[8] = q2.x; x[9] = q2.y; x[10] = q2.z; x[11] = q2.w;
    } else {                                     // the end of a row or of the matrix
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
            v.w[i] = lo | (hi << 16);
        }
        return v;
    }
    return shifted(x, off);
}

// 16 bf16 values to p, n of them valid.  The whole warp calls it, its lanes' columns following one another.
template <bool WIDE>
__device__ __forceinline__ void store16(uint16_t* p, const V16& v, int64_t n) {
    if (WIDE) {
        if (n >= 16) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]),
                         "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
                         : "memory");
            return;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < n) p[i] = (uint16_t)(v.w[i >> 1] >> ((i & 1) * 16));
        return;
    }
    const int lane = threadIdx.x & 31;
    const uint32_t off = (uint32_t)((uintptr_t)p & 15);          // the same in every lane: they are 32 bytes apart
    const bool whole = n >= 16;
    const bool joined = __shfl_down_sync(~0u, (int)whole, 1) && whole && lane < 31;      // writes into the next lane's columns
    const bool covered = __shfl_up_sync(~0u, (int)joined, 1) && lane > 0;                // the lane before wrote this one's first
    uint32_t x[12];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v.w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[8 + i] = __shfl_down_sync(~0u, v.w[i], 1);
    const int head = off ? (16 - (int)off) >> 1 : 0;             // elements before the first aligned chunk
    if (head & 4) {
#pragma unroll
        for (int i = 0; i < 10; ++i) x[i] = x[i + 2];
    }
    if (head & 2) {
#pragma unroll
        for (int i = 0; i < 9; ++i) x[i] = x[i + 1];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], (head & 1) * 16);
    const bool second = joined || head == 0;
    if (whole) {
        *reinterpret_cast<uint4*>(p + head) = make_uint4(x[0], x[1], x[2], x[3]);
        if (second) *reinterpret_cast<uint4*>(p + head + 8) = make_uint4(x[4], x[5], x[6], x[7]);
    }
    // what is left: the elements before the first chunk and after the last, or all of a row's last few
    if (whole) {
        if (!covered && head) {
            const uint32_t sh = (head & 1) * 16;
            const uint32_t y[3] = {__funnelshift_r(v.w[0], v.w[1], sh), __funnelshift_r(v.w[1], v.w[2], sh), __funnelshift_r(v.w[2], v.w[3], sh)};
            if (head & 1) p[0] = (uint16_t)v.w[0];
            if (head & 2) *reinterpret_cast<uint32_t*>(p + (head & 1)) = y[0];
            if (head & 4) *reinterpret_cast<uint2*>(p + (head & 3)) = (head & 2) ? make_uint2(y[1], y[2]) : make_uint2(y[0], y[1]);
        }
        if (!second) {
            const int left = 8 - head;
            uint16_t* o = p + head + 8;
            if (left & 4) *reinterpret_cast<uint2*>(o) = make_uint2(x[4], x[5]);
            if (left & 2) *reinterpret_cast<uint32_t*>(o + (left & 4)) = (left & 4) ? x[6] : x[4];
            if (left & 1) o[left - 1] = (uint16_t)((left & 4) ? (left & 2 ? x[7] : x[6]) : (left & 2 ? x[5] : x[4]));
        }
    } else if (n > 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < n) p[i] = (uint16_t)(v.w[i >> 1] >> ((i & 1) * 16));
    }
}

__device__ __forceinline__ float2 pair_of(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

// A block of 128 columns held by 8 neighbouring lanes, 16 columns each (f; those past the row's end 0), in the
// format: the thread's codes, and the block's scale byte.  The whole warp calls it.
__device__ __forceinline__ uint4 code16(float2 (&f)[8], uint32_t& byte) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = q8_top2(top, f[i]);
    if (isinf(top)) {
        top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = make_float2(q8_no_inf(f[i].x), q8_no_inf(f[i].y));
            top = q8_top2(top, f[i]);
        }
    }
#pragma unroll
    for (int k = 1; k < 8; k <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
    byte = q8_scale_byte(top);
    const float2 inv = make_float2(q8_inverse(byte), q8_inverse(byte));
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 a = q8_mul2(f[2 * k], inv), b = q8_mul2(f[2 * k + 1], inv);
        w[k] = q8_pack4(a.x, a.y, b.x, b.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// A thread's codes (n of the 16 valid) and its block's scale to their place.
__device__ __forceinline__ void store_code16(const uint4& w, uint32_t byte, int64_t n, const Q8& q, int64_t row, int64_t col) {
    if (n <= 0) return;
    store_codes(q.codes + row * q.ld + col, w, n < 16 ? (int)n : 16);
    if ((col & 127) == 0) q.scales[row * q.lds + (col >> 7)] = (uint8_t)byte;
}
__device__ __forceinline__ void encode16(float2 (&f)[8], int64_t n, const Q8& q, int64_t row, int64_t col) {
    uint32_t byte;
    const uint4 w = code16(f, byte);
    store_code16(w, byte, n, q, row, col);
}

}  // namespace zs
