// The 8-bit format of the training operators (include/zs.h, zs_q8): e4m3 codes with one power-of-two
// scale byte per row and block of 128 columns.  Device helpers to read and write it, and the argument
// checks that its host entry points share.
#pragma once

#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <string>

#include "device.cuh"
#include "plan.h"
#include "trace.h"

namespace zs {

// A zs_q8 with typed pointers, as kernels take it; codes == nullptr: not wanted.
struct Q8 {
    uint8_t* codes;
    uint8_t* scales;
    int64_t ld, lds;
};

// ------------------------------------------------------------------ scales

// Biased exponent of the block scale for a largest finite magnitude `top`: the smallest e >= -127
// with top <= 448 * 2^e, plus 127.  448 = 1.75 * 2^8, so with top = 1.f * 2^E the answer is E - 8
// when 1.f <= 1.75 and E - 7 above; adding 0x1fffff to the bits carries into the exponent exactly
// when the mantissa exceeds 0x600000 (1.75).  Zeros and fp32 subnormals give byte 0.
__device__ __forceinline__ uint32_t q8_scale_byte(float top) {
    const int b = (int)((__float_as_uint(top) + 0x1fffffu) >> 23) - 8;
    return (uint32_t)(b < 0 ? 0 : b);
}
// 2^-e for the scale byte e + 127 (byte <= 247 in every encoded block).
__device__ __forceinline__ float q8_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^e for any scale byte: byte 0 is the fp32 subnormal 2^-127, byte 255 is NaN.
__device__ __forceinline__ float q8_scale(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fffffffu : byte << 23);
}

// ------------------------------------------------------------------ codes

// Two fp32 values -> two e4m3 bytes (lo in bits 0-7), to nearest even, saturating; NaN -> 0x7f.
__device__ __forceinline__ uint32_t q8_pack2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d) {
    return q8_pack2(a, b) | (q8_pack2(c, d) << 16);
}
// Two e4m3 bytes -> two fp32 values (exact: every e4m3 value is an f16 value).
__device__ __forceinline__ float2 q8_unpack2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ void q8_unpack4(uint32_t four, float scale, float* f) {
    const float2 a = q8_unpack2(four & 0xffffu), b = q8_unpack2(four >> 16);
    f[0] = a.x * scale; f[1] = a.y * scale; f[2] = b.x * scale; f[3] = b.y * scale;
}

// max(top, |x|) where x is finite or NaN (NaN never wins); an infinity shows as top = inf.
__device__ __forceinline__ float q8_top(float top, float x) { return fmaxf(top, fabsf(x)); }
// max(top, |x|, |y|) the same way, in one instruction.
__device__ __forceinline__ float q8_top2(float top, float2 x) {
    float d;
    asm("{\n\t.reg .f32 a, b;\n\tabs.f32 a, %2;\n\tabs.f32 b, %3;\n\tmax.f32 %0, %1, a, b;\n\t}" : "=f"(d) : "f"(top), "f"(x.x), "f"(x.y));
    return d;
}
// The encoding's treatment of infinities: NaN in their place.
__device__ __forceinline__ float q8_no_inf(float x) { return isinf(x) ? __uint_as_float(0x7fffffffu) : x; }

// ------------------------------------------------------------------ two values at a time

__device__ __forceinline__ float2 q8_mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 q8_add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 q8_fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// sigmoid(x) = 1 / (1 + 2^(-x log2 e)), two at a time.  The hardware's power of two and reciprocal flush
// what is subnormal to 0: 2^y there stands beside 1, and a sigmoid there is below 2^-126.  Their errors and
// that of the rounded exponent are within 2^-18 of the sigmoid for |x| <= 32, 13 bits below an e4m3 step.
__device__ __forceinline__ float2 q8_sigmoid2(float2 x) {
    const float2 y = q8_mul2(x, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(y.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(y.y));
    e = q8_fma2(e, make_float2(1.f, 1.f), make_float2(1.f, 1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
    return e;
}

// ------------------------------------------------------------------ host checks

namespace q8_host {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 256;

inline int fail(const char* fn, const std::string& what) {
    set_error(std::string(fn) + ": " + what);
    return ZS_ERR_INVALID;
}

inline int cuda_status(const char* fn, cudaError_t e) {
    if (e == cudaSuccess) return ZS_OK;
    set_error(std::string(fn) + ": " + cudaGetErrorString(e));
    return ZS_ERR_CUDA;
}

inline int check_dim(const char* fn, const char* name, int64_t v, int64_t least) {
    if (v < least || v > kMaxDim) return fail(fn, std::string(name) + " out of range");
    return ZS_OK;
}

// A bf16 matrix: 2-byte aligned, rows ld >= cols elements apart.  An empty one may be NULL.
inline int check_bf16(const char* fn, const char* name, const void* p, int64_t ld, int64_t rows, int64_t cols) {
    if (!p && rows > 0 && cols > 0) return fail(fn, std::string(name) + " is NULL");
    if ((uintptr_t)p & 1) return fail(fn, std::string(name) + " is not 2-byte aligned");
    if (ld < cols || ld > (int64_t(1) << 38)) return fail(fn, std::string(name) + ": row distance out of range");
    return ZS_OK;
}

// A zs_q8 into its typed form; NULL is allowed when `optional` and gives codes == nullptr.  An empty
// matrix may have NULL pointers.
inline int check_q8(const char* fn, const char* name, const zs_q8* q, int64_t rows, int64_t cols, bool optional, Q8* out) {
    *out = Q8{nullptr, nullptr, 0, 0};
    if (!q) return optional ? ZS_OK : fail(fn, std::string(name) + " is NULL");
    if ((!q->codes || !q->scales) && rows > 0 && cols > 0) return fail(fn, std::string(name) + ": codes / scales is NULL");
    if ((uintptr_t)q->codes & 15) return fail(fn, std::string(name) + ": codes are not 16-byte aligned");
    if (q->ld < cols || (q->ld & 15) || q->ld > (int64_t(1) << 38))
        return fail(fn, std::string(name) + ": ld must be a multiple of 16 and at least the columns");
    if (q->ld_scales < (cols + ZS_Q8_BLOCK - 1) / ZS_Q8_BLOCK || q->ld_scales > (int64_t(1) << 38))
        return fail(fn, std::string(name) + ": ld_scales is smaller than the blocks of a row");
    *out = Q8{(uint8_t*)q->codes, (uint8_t*)q->scales, q->ld, q->ld_scales};
    return ZS_OK;
}

// Whether accesses of `bytes` (16 or 32) of a bf16 matrix's rows are aligned.
inline bool wide(const void* p, int64_t ld, int bytes = 16) { return ((uintptr_t)p & (bytes - 1)) == 0 && (ld & (bytes / 2 - 1)) == 0; }

inline int sm_count() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
    cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace q8_host

#define ZS_Q8_TRY(x)                       \
    do {                                   \
        const int rc_ = (x);               \
        if (rc_ != ZS_OK) return rc_;      \
    } while (0)

}  // namespace zs
