// RMS norm with the residual's addition and the gated activation, forward to 8 bits and backward from
// what was kept in 8 bits.  Everything here moves bytes: a value is read once and every output written
// once, with the row or block statistics between the two in registers.
#include "q8_tile.cuh"

namespace zs {

namespace {

// ------------------------------------------------------------------ vectors of 8 columns

// 8 bf16 values at p, n (<= 8) of them valid, the others 0.
template <bool WIDE>
__device__ __forceinline__ uint4 load8(const uint16_t* p, int n) {
    if (n <= 0) return make_uint4(0, 0, 0, 0);
    if (WIDE && n >= 8) return __ldcs(reinterpret_cast<const uint4*>(p));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
        w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool WIDE>
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8], int n) {
    if (n <= 0) return;
    const BfVec<8> v = pack(f);
    if (WIDE && n >= 8) {
        __stcs(reinterpret_cast<uint4*>(p), v.w);
        return;
    }
    const uint32_t w[4] = {v.w.x, v.w.y, v.w.z, v.w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint16_t)(w[i >> 1] >> ((i & 1) * 16));
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) { unpack(BfVec<8>{w}, f); }

// Encodes a block of 128 columns held by 16 neighbouring lanes, 8 columns each (f, n of them valid,
// the others 0): the whole warp calls it.
__device__ __forceinline__ void encode8(float (&f)[8], int n, const Q8& q, int64_t row, int64_t col) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = q8_top(top, f[i]);
    if (isinf(top)) {
        top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = q8_no_inf(f[i]);
            top = q8_top(top, f[i]);
        }
    }
#pragma unroll
    for (int k = 1; k < 16; k <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
    const uint32_t byte = q8_scale_byte(top);
    const float inv = q8_inverse(byte);
    const uint2 w = make_uint2(q8_pack4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                               q8_pack4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
    if (n <= 0) return;
    uint8_t* p = q.codes + row * q.ld + col;
    if (n >= 8) {
        __stcs(reinterpret_cast<uint2*>(p), w);
    } else {
        for (int i = 0; i < n; ++i) p[i] = (uint8_t)((i < 4 ? w.x : w.y) >> ((i & 3) * 8));
    }
    if ((col & 127) == 0) q.scales[row * q.lds + (col >> 7)] = (uint8_t)byte;
}

// Sum over the CTA's threads, the same bits in every thread; `sh` holds one float per warp and is free
// again once every thread has passed a later barrier.
__device__ __forceinline__ float block_sum(float x, float* sh) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(~0u, x, k);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    float sum = 0.f;
    for (int k = 0; k < warps; ++k) sum += sh[k];
    return sum;
}

// a + b and its rounding error, exactly.
__device__ __forceinline__ float2 two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}

// Sum over the CTA's threads with the additions' rounding errors collected beside it, the same bits in
// every thread.
__device__ __forceinline__ float2 block_sum2(float x, float2* sh) {
    float2 v = make_float2(x, 0.f);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        const float2 o = make_float2(__shfl_xor_sync(~0u, v.x, k), __shfl_xor_sync(~0u, v.y, k));
        const float2 s = two_sum(v.x, o.x);
        v = make_float2(s.x, (v.y + o.y) + s.y);
    }
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[0];
    for (int k = 1; k < warps; ++k) {
        const float2 s = two_sum(v.x, sh[k].x);
        v = make_float2(s.x, v.y + sh[k].y + s.y);
    }
    return v;
}

// 1 / sqrt(sum / n + eps) as an fp32 value and what rounding took from it.  An output code goes to its
// neighbour where fp32 rounding carries a value across the middle between two codes; with the factor
// common to a whole row in two words and one rounding per output (norm_output) that is all but gone, at
// a few operations per row.
__device__ __forceinline__ float2 inverse_root(float2 sum, float n, float eps) {
    const float q = __fdiv_rn(sum.x, n);
    const float rest = (fmaf(-q, n, sum.x) + sum.y) / n;
    const float2 v = two_sum(q, eps);
    const float root = __fsqrt_rn(v.x), r = __fdiv_rn(1.f, root);
    // v + rest = root^2 + d and 1 / root = r (1 + e): 1 / sqrt(v + rest) = r (1 + e - d / (2 root^2))
    const float d = (v.y + rest) - fmaf(root, root, -v.x), e = fmaf(-r, root, 1.f);
    const float part = e - 0.5f * d * r * r, hi = fmaf(r, part, r);
    if (!(isfinite(hi) && hi > 0.f)) return make_float2(r, 0.f);       // sums of 0, infinity or NaN
    return make_float2(hi, fmaf(r, part, r - hi));
}

// t * r * w rounded once, and where that lands exactly on what may be the middle between two codes
// (the low 19 bits of the mantissa are 0), moved by one bit to the side of the unrounded product.
__device__ __forceinline__ float norm_output(float t, float2 r, float w) {
    const float p = t * r.x, rest = fmaf(t, r.x, -p) + t * r.y;
    const float y = fmaf(p, w, rest * w);
    if ((__float_as_uint(y) & 0x7ffffu) == 0 && y != 0.f && isfinite(y)) {
        const float off = fmaf(p, w, -y) + rest * w;
        if (off != 0.f) return __uint_as_float(__float_as_uint(y) + ((off > 0.f) == (y > 0.f) ? 1 : -1));
    }
    return y;
}

// ------------------------------------------------------------------ norm, forward

struct NormArgs {
    const uint16_t *x, *res, *weight;
    int64_t ldx, ldr, lds, rows, cols;
    float eps;
    Q8 y, s_q8;
    uint16_t* s;
    float* rstd;
};

// One CTA per row.  NV > 0: the row's sum stays in registers, NV vectors of 8 columns per thread.
// NV = 0, for rows longer than registers hold: the row is read a second time (from L2).
template <int NV, bool WIDE>
__global__ void __launch_bounds__(512) k_rmsnorm_q8(const __grid_constant__ NormArgs a) {
    __shared__ float2 sh[32];
    dependent_launch_prologue();
    const int64_t row = blockIdx.x;
    const uint16_t* x = a.x + row * a.ldx;
    const uint16_t* res = a.res ? a.res + row * a.ldr : nullptr;
    const int64_t step = (int64_t)blockDim.x * 8, col0 = (int64_t)threadIdx.x * 8;
    auto valid = [&](int64_t c) { return (int)(a.cols - c < 8 ? a.cols - c : 8); };
    auto sum_at = [&](int64_t c, float (&t)[8]) {
        const int n = valid(c);
        const uint4 wx = load8<WIDE>(x + c, n);
        unpack8(wx, t);
        if (res) {
            float r[8];
            unpack8(load8<WIDE>(res + c, n), r);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] += r[i];
        }
    };
    auto squares = [](const float (&t)[8]) {
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) q = fmaf(t[i], t[i], q);
        return q;
    };
    auto write = [&](int64_t c, float (&t)[8], float2 r) {
        const int n = valid(c);
        float w[8], y[8];
        unpack8(load8<WIDE>(a.weight + c, n), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = norm_output(t[i], r, w[i]);
        encode8(y, n, a.y, row, c);
        if (a.s) store8<WIDE>(a.s + row * a.lds + c, t, n);
        if (a.s_q8.codes) encode8(t, n, a.s_q8, row, c);
    };
    float sq = 0.f;
    if constexpr (NV > 0) {
        float t[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            sum_at(col0 + v * step, t[v]);
            sq += squares(t[v]);
        }
        const float2 r = inverse_root(block_sum2(sq, sh), (float)a.cols, a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (v * step < a.cols) write(col0 + v * step, t[v], r);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = r.x;
    } else {
        float t[8];
        for (int64_t c = col0; c - col0 < a.cols; c += step) {
            sum_at(c, t);
            sq += squares(t);
        }
        const float2 r = inverse_root(block_sum2(sq, sh), (float)a.cols, a.eps);
        for (int64_t c = col0; c - col0 < a.cols; c += step) {
            sum_at(c, t);
            write(c, t, r);
        }
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = r.x;
    }
}

// ------------------------------------------------------------------ norm, backward

struct NormBackArgs {
    const uint16_t *dy, *s, *weight, *ds;
    Q8 s_q8;
    const float* rstd;
    uint16_t* dx;
    float* partials;
    int64_t lddy, lds, ldds, lddx, rows, cols;
};

// Each CTA takes rows blockIdx.x, + gridDim.x, ... and keeps its part of dw: thread t owns the columns
// of its vectors in every row, in registers (NV > 0) or in its row of `partials` (NV = 0).
template <int NV, bool WIDE>
__global__ void __launch_bounds__(512) k_rmsnorm_backward(const __grid_constant__ NormBackArgs a) {
    __shared__ float sh[2][32];
    dependent_launch_prologue();
    constexpr int N1 = NV > 0 ? NV : 1;
    const int64_t step = (int64_t)blockDim.x * 8, col0 = (int64_t)threadIdx.x * 8;
    auto valid = [&](int64_t c) { return (int)(a.cols - c < 8 ? a.cols - c : 8); };
    // dy and the normalised sum of 8 columns
    auto inputs = [&](int64_t row, int64_t c, float r, float (&dy)[8], float (&xh)[8]) {
        const int n = valid(c);
        unpack8(load8<WIDE>(a.dy + row * a.lddy + c, n), dy);
        if (a.s_q8.codes) {
            const uint8_t* p = a.s_q8.codes + row * a.s_q8.ld + c;
            uint2 w = make_uint2(0, 0);
            float q = 0.f;
            if (n > 0) q = q8_scale(a.s_q8.scales[row * a.s_q8.lds + (c >> 7)]);
            if (n >= 8) {
                w = __ldcs(reinterpret_cast<const uint2*>(p));
            } else {
                for (int i = 0; i < n; ++i) (i < 4 ? w.x : w.y) |= (uint32_t)p[i] << ((i & 3) * 8);
            }
            q8_unpack4(w.x, q, xh);
            q8_unpack4(w.y, q, xh + 4);
        } else {
            unpack8(load8<WIDE>(a.s + row * a.lds + c, n), xh);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[i] *= r;
    };
    auto weight_at = [&](int64_t c, float (&w)[8]) { unpack8(load8<WIDE>(a.weight + c, valid(c)), w); };
    auto dot = [](const float (&dy)[8], const float (&w)[8], const float (&xh)[8]) {
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) d = fmaf(dy[i] * w[i], xh[i], d);
        return d;
    };
    auto write = [&](int64_t row, int64_t c, float r, float along, const float (&dy)[8], const float (&w)[8],
                     const float (&xh)[8]) {
        const int n = valid(c);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = r * (dy[i] * w[i] - xh[i] * along);
        if (a.ds) {
            float d[8];
            unpack8(load8<WIDE>(a.ds + row * a.ldds + c, n), d);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += d[i];
        }
        store8<WIDE>(a.dx + row * a.lddx + c, o, n);
    };
    const float inv_cols = 1.f / (float)a.cols;
    float* part = a.partials + (int64_t)blockIdx.x * a.cols;
    float dw[N1][8];
#pragma unroll
    for (int v = 0; v < N1; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
    int turn = 0;
    bool first = true;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1, first = false) {
        const float r = a.rstd[row];
        float d = 0.f;
        if constexpr (NV > 0) {
            float dy[NV][8], xh[NV][8], w[8];
#pragma unroll
            for (int v = 0; v < NV; ++v) inputs(row, col0 + v * step, r, dy[v], xh[v]);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                weight_at(col0 + v * step, w);
                d += dot(dy[v], w, xh[v]);
            }
            const float along = block_sum(d, sh[turn]) * inv_cols;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                weight_at(col0 + v * step, w);
                write(row, col0 + v * step, r, along, dy[v], w, xh[v]);
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[v][i] = fmaf(dy[v][i], xh[v][i], dw[v][i]);
            }
        } else {
            float dy[8], xh[8], w[8];
            for (int64_t c = col0; c < a.cols; c += step) {
                inputs(row, c, r, dy, xh);
                weight_at(c, w);
                d += dot(dy, w, xh);
            }
            const float along = block_sum(d, sh[turn]) * inv_cols;
            for (int64_t c = col0; c < a.cols; c += step) {
                inputs(row, c, r, dy, xh);
                weight_at(c, w);
                write(row, c, r, along, dy, w, xh);
                const int n = valid(c);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < n) part[c + i] = fmaf(dy[i], xh[i], first ? 0.f : part[c + i]);
            }
        }
    }
    if constexpr (NV > 0) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t c = col0 + v * step;
            const int n = valid(c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) part[c + i] = dw[v][i];
        }
    }
}

// dw from the partial sums: a CTA takes 32 columns, its 8 warps a share of the partials each, added in
// index order within a warp and over the warps.
__global__ void __launch_bounds__(256) k_rmsnorm_dw(const float* partials, int64_t count, int64_t cols, uint16_t* dw,
                                                    float scale, int first) {
    __shared__ float sh[8][32];
    dependent_launch_prologue();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < cols)
        for (int64_t k = warp; k < count; k += 8) sum += partials[k * cols + c];
    sh[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < cols) {
        float all = sh[0][lane];
#pragma unroll
        for (int k = 1; k < 8; ++k) all += sh[k][lane];
        all *= scale;
        if (!first) all += bf16_to_f32(dw[c]);
        dw[c] = f32_to_bf16(all);
    }
}

// ------------------------------------------------------------------ gated activation

struct GateArgs {
    const uint16_t *gate, *up;
    int64_t ldg, ldu, rows, cols;
    Q8 h, gate_q, up_q;
};

constexpr int kGateThreads = 128;

// A CTA takes 1024 columns of a row, 8 per thread.
template <bool WIDE>
__global__ void __launch_bounds__(kGateThreads) k_swiglu_q8(const __grid_constant__ GateArgs a) {
    dependent_launch_prologue();
    const int64_t row = blockIdx.x, c = ((int64_t)blockIdx.y * kGateThreads + threadIdx.x) * 8;
    const int n = (int)(a.cols - c < 8 ? a.cols - c : 8);
    const uint4 wg = load8<WIDE>(a.gate + row * a.ldg + c, n), wu = load8<WIDE>(a.up + row * a.ldu + c, n);
    float g[8], u[8], h[8];
    unpack8(wg, g);
    unpack8(wu, u);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 x = make_float2(g[i], g[i + 1]);
        const float2 y = q8_mul2(q8_mul2(x, q8_sigmoid2(x)), make_float2(u[i], u[i + 1]));
        h[i] = y.x;
        h[i + 1] = y.y;
    }
    encode8(h, n, a.h, row, c);
    if (a.gate_q.codes) encode8(g, n, a.gate_q, row, c);
    if (a.up_q.codes) encode8(u, n, a.up_q, row, c);
}

// Threads and register vectors for a row of `cols` columns: the fewest vectors per thread that keep the
// CTA within `most` threads; nv = 0 when the row does not fit in registers.
void row_shape(int64_t cols, int most, int* threads, int* nv) {
    const int64_t vecs = (cols + 7) / 8;
    for (int k = 1; k <= 4; k *= 2) {
        const int64_t need = ((vecs + k - 1) / k + 31) / 32 * 32;
        if (need <= most) {
            *threads = (int)need;
            *nv = k;
            return;
        }
    }
    *threads = 512;
    *nv = 0;
}

template <bool WIDE>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
    int threads, nv;
    row_shape(a.cols, 512, &threads, &nv);
    const dim3 grid((unsigned)a.rows), block(threads);
    switch (nv) {
        case 1: return launch_kernel(k_rmsnorm_q8<1, WIDE>, grid, block, 0, st, a);
        case 2: return launch_kernel(k_rmsnorm_q8<2, WIDE>, grid, block, 0, st, a);
        case 4: return launch_kernel(k_rmsnorm_q8<4, WIDE>, grid, block, 0, st, a);
        default: return launch_kernel(k_rmsnorm_q8<0, WIDE>, grid, block, 0, st, a);
    }
}

template <bool WIDE>
cudaError_t launch_norm_back(const NormBackArgs& a, int parts, cudaStream_t st) {
    int threads, nv;
    row_shape(a.cols, 512, &threads, &nv);
    const dim3 grid((unsigned)parts), block(threads);
    switch (nv) {
        case 1: return launch_kernel(k_rmsnorm_backward<1, WIDE>, grid, block, 0, st, a);
        case 2: return launch_kernel(k_rmsnorm_backward<2, WIDE>, grid, block, 0, st, a);
        case 4: return launch_kernel(k_rmsnorm_backward<4, WIDE>, grid, block, 0, st, a);
        default: return launch_kernel(k_rmsnorm_backward<0, WIDE>, grid, block, 0, st, a);
    }
}

}  // namespace

}  // namespace zs

using namespace zs::q8_host;

extern "C" int zs_rmsnorm_q8(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                             float eps, int64_t rows, int64_t cols, const zs_q8* y, void* s, int64_t lds,
                             const zs_q8* s_q8, float* rstd, void* stream) {
    static const char* fn = "zs_rmsnorm_q8";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::NormArgs a{};
    ZS_Q8_TRY(check_dim(fn, "rows", rows, 0));
    ZS_Q8_TRY(check_dim(fn, "cols", cols, 1));
    ZS_Q8_TRY(check_bf16(fn, "x", x, ldx, rows, cols));
    if (residual) ZS_Q8_TRY(check_bf16(fn, "residual", residual, ldr, rows, cols));
    ZS_Q8_TRY(check_bf16(fn, "weight", weight, cols, 1, cols));
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(fn, "eps must be finite and not negative");
    ZS_Q8_TRY(check_q8(fn, "y", y, rows, cols, false, &a.y));
    if (s) ZS_Q8_TRY(check_bf16(fn, "s", s, lds, rows, cols));
    ZS_Q8_TRY(check_q8(fn, "s_q8", s_q8, rows, cols, true, &a.s_q8));
    if ((uintptr_t)rstd & 3) return fail(fn, "rstd is not 4-byte aligned");
    if (rows == 0) return ZS_OK;
    a.x = (const uint16_t*)x;
    a.res = (const uint16_t*)residual;
    a.weight = (const uint16_t*)weight;
    a.ldx = ldx;
    a.ldr = ldr;
    a.lds = lds;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.s = (uint16_t*)s;
    a.rstd = rstd;
    const bool w = wide(x, ldx) && (!residual || wide(residual, ldr)) && wide(weight, 0) && (!s || wide(s, lds));
    const cudaStream_t st = (cudaStream_t)stream;
    return cuda_status(fn, w ? zs::launch_norm<true>(a, st) : zs::launch_norm<false>(a, st));
}

extern "C" int zs_rmsnorm_backward(const void* dy, int64_t lddy, const void* s, int64_t lds, const zs_q8* s_q8,
                                   const void* weight, const float* rstd, const void* ds, int64_t ldds, int64_t rows,
                                   int64_t cols, void* dx, int64_t lddx, void* dw, float scale, int32_t first,
                                   float* partials, int64_t n_partials, void* stream) {
    static const char* fn = "zs_rmsnorm_backward";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::NormBackArgs a{};
    ZS_Q8_TRY(check_dim(fn, "rows", rows, 0));
    ZS_Q8_TRY(check_dim(fn, "cols", cols, 1));
    ZS_Q8_TRY(check_bf16(fn, "dy", dy, lddy, rows, cols));
    if ((s && s_q8) || (!s && !s_q8 && rows > 0)) return fail(fn, "exactly one of s and s_q8 must be given");
    if (s) ZS_Q8_TRY(check_bf16(fn, "s", s, lds, rows, cols));
    ZS_Q8_TRY(check_q8(fn, "s_q8", s_q8, rows, cols, true, &a.s_q8));
    ZS_Q8_TRY(check_bf16(fn, "weight", weight, cols, 1, cols));
    if ((!rstd && rows > 0) || ((uintptr_t)rstd & 3)) return fail(fn, "rstd is NULL or not 4-byte aligned");
    if (ds) ZS_Q8_TRY(check_bf16(fn, "ds", ds, ldds, rows, cols));
    ZS_Q8_TRY(check_bf16(fn, "dx", dx, lddx, rows, cols));
    ZS_Q8_TRY(check_bf16(fn, "dw", dw, cols, 1, cols));
    if (!std::isfinite(scale)) return fail(fn, "scale must be finite");
    if (!partials || ((uintptr_t)partials & 15)) return fail(fn, "partials is NULL or not 16-byte aligned");
    if (n_partials < 1) return fail(fn, "n_partials must be at least 1");
    a.dy = (const uint16_t*)dy;
    a.s = (const uint16_t*)s;
    a.weight = (const uint16_t*)weight;
    a.ds = (const uint16_t*)ds;
    a.rstd = rstd;
    a.dx = (uint16_t*)dx;
    a.partials = partials;
    a.lddy = lddy;
    a.lds = lds;
    a.ldds = ldds;
    a.lddx = lddx;
    a.rows = rows;
    a.cols = cols;
    const bool w = wide(dy, lddy) && (!s || wide(s, lds)) && wide(weight, 0) && (!ds || wide(ds, ldds)) && wide(dx, lddx);
    const cudaStream_t st = (cudaStream_t)stream;
    int64_t parts = 2 * (int64_t)sm_count();
    if (parts > n_partials) parts = n_partials;
    if (parts > ZS_Q8_MAX_PARTIALS) parts = ZS_Q8_MAX_PARTIALS;
    if (parts > rows) parts = rows;
    if (parts > 0)
        ZS_Q8_TRY(cuda_status(fn, w ? zs::launch_norm_back<true>(a, (int)parts, st)
                                    : zs::launch_norm_back<false>(a, (int)parts, st)));
    return cuda_status(fn, zs::launch_kernel(zs::k_rmsnorm_dw, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, st,
                                             (const float*)partials, parts, cols, (uint16_t*)dw, scale, (int)first));
}

extern "C" int zs_swiglu_q8(const void* gate, int64_t ldg, const void* up, int64_t ldu, int64_t rows, int64_t cols,
                            const zs_q8* h, const zs_q8* gate_q, const zs_q8* up_q, void* stream) {
    static const char* fn = "zs_swiglu_q8";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::GateArgs a{};
    ZS_Q8_TRY(check_dim(fn, "rows", rows, 0));
    ZS_Q8_TRY(check_dim(fn, "cols", cols, 1));
    ZS_Q8_TRY(check_bf16(fn, "gate", gate, ldg, rows, cols));
    ZS_Q8_TRY(check_bf16(fn, "up", up, ldu, rows, cols));
    ZS_Q8_TRY(check_q8(fn, "h", h, rows, cols, false, &a.h));
    ZS_Q8_TRY(check_q8(fn, "gate_q", gate_q, rows, cols, true, &a.gate_q));
    ZS_Q8_TRY(check_q8(fn, "up_q", up_q, rows, cols, true, &a.up_q));
    if (rows == 0) return ZS_OK;
    a.gate = (const uint16_t*)gate;
    a.up = (const uint16_t*)up;
    a.ldg = ldg;
    a.ldu = ldu;
    a.rows = rows;
    a.cols = cols;
    const int64_t pieces = (cols + zs::kGateThreads * 8 - 1) / (zs::kGateThreads * 8);
    if (pieces > 65535) return fail(fn, "cols too large for one launch");
    const dim3 grid((unsigned)rows, (unsigned)pieces), block(zs::kGateThreads);
    const cudaStream_t st = (cudaStream_t)stream;
    return cuda_status(fn, wide(gate, ldg) && wide(up, ldu) ? zs::launch_kernel(zs::k_swiglu_q8<true>, grid, block, 0, st, a)
                                                            : zs::launch_kernel(zs::k_swiglu_q8<false>, grid, block, 0, st, a));
}

extern "C" int zs_swiglu_backward_q8(const void* dh, int64_t lddh, const zs_q8* gate_q, const zs_q8* up_q,
                                     int64_t rows, int64_t cols, const zs_q8* dgate, const zs_q8* dup,
                                     const zs_q8* dgate_t, const zs_q8* dup_t, const zs_q8* h_t, void* stream) {
    static const char* fn = "zs_swiglu_backward_q8";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::TileArgs a{};
    ZS_Q8_TRY(check_dim(fn, "rows", rows, 0));
    ZS_Q8_TRY(check_dim(fn, "cols", cols, 1));
    ZS_Q8_TRY(check_bf16(fn, "dh", dh, lddh, rows, cols));
    ZS_Q8_TRY(check_q8(fn, "gate_q", gate_q, rows, cols, false, &a.a));
    ZS_Q8_TRY(check_q8(fn, "up_q", up_q, rows, cols, false, &a.b));
    ZS_Q8_TRY(check_q8(fn, "dgate", dgate, rows, cols, true, &a.rows_out[0]));
    ZS_Q8_TRY(check_q8(fn, "dup", dup, rows, cols, true, &a.rows_out[1]));
    ZS_Q8_TRY(check_q8(fn, "dgate_t", dgate_t, cols, rows, true, &a.cols_out[0]));
    ZS_Q8_TRY(check_q8(fn, "dup_t", dup_t, cols, rows, true, &a.cols_out[1]));
    ZS_Q8_TRY(check_q8(fn, "h_t", h_t, cols, rows, true, &a.cols_out[2]));
    if (!dgate && !dup && !dgate_t && !dup_t && !h_t) return fail(fn, "every output is NULL");
    if (rows == 0) return ZS_OK;
    a.x = (const uint16_t*)dh;
    a.ldx = lddh;
    a.rows = rows;
    a.cols = cols;
    const cudaStream_t st = (cudaStream_t)stream;
    return cuda_status(fn, wide(dh, lddh) ? zs::launch_tiles<zs::kTileGate, true>(a, st) : zs::launch_tiles<zs::kTileGate, false>(a, st));
}
