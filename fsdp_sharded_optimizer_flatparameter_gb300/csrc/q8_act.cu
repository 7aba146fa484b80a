// RMS norm with the residual's addition and the gated activation, forward to 8 bits and backward from
// what was kept in 8 bits.  Everything here moves bytes: a value is read once and every output written
// once, with the row or block statistics between the two in registers.
#include "q8_tile.cuh"

namespace zs {

namespace {

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

constexpr int kSlotStages = 2;       // rows under way

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

// Encodes a block of 128 columns held by 8 neighbouring lanes, 16 columns each (f; n of them valid, the others
// 0): the whole warp calls it.
__device__ __forceinline__ void encode16(float2 (&f)[8], int64_t n, const Q8& q, int64_t row, int64_t col) {
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
    const uint32_t byte = q8_scale_byte(top);
    const float2 inv = make_float2(q8_inverse(byte), q8_inverse(byte));
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 a = q8_mul2(f[2 * k], inv), b = q8_mul2(f[2 * k + 1], inv);
        w[k] = q8_pack4(a.x, a.y, b.x, b.y);
    }
    if (n <= 0) return;
    store_codes(q.codes + row * q.ld + col, make_uint4(w[0], w[1], w[2], w[3]), n < 16 ? (int)n : 16);
    if ((col & 127) == 0) q.scales[row * q.lds + (col >> 7)] = (uint8_t)byte;
}

// Sum over the `threads` threads of the caller's group (whole warps; barrier `id` is the group's own), the same
// bits in every thread; `sh` holds one float per warp and is free again once every thread of the group has
// passed a later barrier.
__device__ __forceinline__ float group_sum(float x, float* sh, int threads, int id) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(~0u, x, k);
    const int warps = threads >> 5, warp = (threadIdx.x >> 5) % warps;
    if (warps == 1) return x;
    if ((threadIdx.x & 31) == 0) sh[warp] = x;
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
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
    if (warps == 1) return v;
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
// common to a whole row in two words and one rounding per output (norm_outputs) that is all but gone, at
// a few operations per row: one Newton step on the hardware's reciprocal root, whose residual
// 1 - (v + rest) r^2 is taken from exact products.
__device__ __forceinline__ float2 inverse_root(float2 sum, float n, float inv_n, float eps) {
    const float q = sum.x * inv_n;
    const float2 v = two_sum(q, eps);
    const float rest = v.y + (fmaf(-q, n, sum.x) + sum.y) * inv_n;
    const float r = rsqrtf(v.x);
    const float h = v.x * r, hl = fmaf(v.x, r, -h);
    const float off = fmaf(-h, r, 1.f) - (hl + rest * r) * r;
    const float hi = fmaf(0.5f * r, off, r);
    if (!(isfinite(hi) && hi > 0.f)) return make_float2(r, 0.f);       // sums of 0, infinity or NaN
    return make_float2(hi, fmaf(0.5f * r, off, r - hi));
}

// t * r * w rounded once, and where that lands exactly on what may be the middle between two codes (the low 19
// bits of the mantissa are 0), moved by one bit to the side of the unrounded product.
__device__ __forceinline__ void norm_outputs(const float2 (&t)[8], float2 r, const V16& weight, float2 (&y)[8]) {
    const float2 hi = make_float2(r.x, r.x), lo = make_float2(r.y, r.y), minus = make_float2(-1.f, -1.f);
    uint32_t low = ~0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 w = pair_of(weight.w[i]);
        const float2 p = q8_mul2(t[i], hi), rest = q8_fma2(t[i], lo, q8_fma2(t[i], hi, q8_mul2(p, minus)));
        y[i] = q8_fma2(p, w, q8_mul2(rest, w));
        low = min(low, min(__float_as_uint(y[i].x) << 13, __float_as_uint(y[i].y) << 13));
    }
    if (low) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 w = pair_of(weight.w[i]);
        auto nudge = [&](float t, float w, float& y) {
            if ((__float_as_uint(y) << 13) != 0 || y == 0.f || !isfinite(y)) return;
            const float p = t * r.x, rest = fmaf(t, r.y, fmaf(t, r.x, -p)), off = fmaf(p, w, -y) + rest * w;
            if (off != 0.f) y = __uint_as_float(__float_as_uint(y) + ((off > 0.f) == (y > 0.f) ? 1 : -1));
        };
        nudge(t[i].x, w.x, y[i].x);
        nudge(t[i].y, w.y, y[i].y);
    }
}

// ------------------------------------------------------------------ rows through shared memory

constexpr int kRowStages = 4;
constexpr int kRowSmem = kRowStages * 8192 * 6;      // the widest row of 512 threads, three bf16 matrices

// bytes (a multiple of 16) from src to dst, both 16-byte aligned, counted on bar.
__device__ __forceinline__ void bulk_row(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(su32(dst)), "l"(src),
                 "r"(bytes), "r"(su32(bar))
                 : "memory");
}
__device__ __forceinline__ V16 row16(const uint8_t* p) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    return V16{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
// After a wait ran out: one thread lets the copies on their way land, so that the CTA may exit.
__device__ __forceinline__ void drain_rows(uint64_t* full, int at, uint32_t parity, int64_t left, unsigned int* error) {
    atomicCAS(error, 0u, ZS_DEVERR_TILE_WAIT);
    for (int i = 0; i < kRowStages && i < left; ++i)
        mbar_wait(full + (at + i) % kRowStages, at + i >= kRowStages ? parity ^ 1 : parity, kDrainLimit);
}

// ------------------------------------------------------------------ norm, forward

struct NormArgs {
    const uint16_t *x, *res, *weight;
    int64_t ldx, ldr, lds, rows, cols;
    float eps, inv_cols;
    Q8 y, s_q8;
    uint16_t* s;
    float* rstd;
};

// A CTA takes rows blockIdx.x, + gridDim.x, ...  NV > 0: a row's sum stays in registers, NV vectors of 16 columns
// per thread, and the next row's loads are under way while a row is reduced and written.  NV = 0, for rows
// longer than that: the row is read a second time (from L2).  Rows brought by bulk copies through shared memory, two
// to four stages of them, took the same time (16384 x 4096: 91-93 us, and 92-95 with 640 to 1024 threads per SM).
template <int NV, bool WIDE>
__global__ void __launch_bounds__(512) k_rmsnorm_q8(const __grid_constant__ NormArgs a) {
    __shared__ float2 sh[2][16];
    dependent_launch_prologue();
    constexpr int N1 = NV > 0 ? NV : 1;
    const int64_t step = (int64_t)blockDim.x * 16, col0 = (int64_t)threadIdx.x * 16;
    const Span sx = span_of(a.x, a.ldx, a.rows, a.cols), sr = span_of(a.res, a.ldr, a.rows, a.cols);
    const Span sw = span_of(a.weight, 0, 1, a.cols);
    auto squares = [](const float2 (&t)[8]) {
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) q = q8_fma2(t[i], t[i], q);
        return q.x + q.y;
    };
    auto sums = [](const V16& x, const V16& r, float2 (&t)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[i] = q8_add2(pair_of(x.w[i]), pair_of(r.w[i]));
        }
    };
    auto write = [&](int64_t row, int64_t c, float2 (&t)[8], float2 r, const V16& w) {
        const int64_t n = a.cols - c;
        float2 y[8];
        norm_outputs(t, r, w, y);
        encode16(y, n, a.y, row, c);
        if (a.s) {
            V16 v;
#pragma unroll
            for (int i = 0; i < 8; ++i) v.w[i] = pack_bf16x2(t[i].x, t[i].y);
            store16<WIDE>(a.s + row * a.lds + c, v, n);
        }
        if (a.s_q8.codes) encode16(t, n, a.s_q8, row, c);
    };
    const V16 zero = {};
    int turn = 0;
    if constexpr (NV > 0) {
        V16 w[N1], x[N1], r[N1];
        extern __shared__ __align__(16) uint8_t slots[];         // [stage][x, res][v][thread], unless WIDE
        auto slot = [&](int at, int m, int v) { return slots + ((int64_t)((at * 2 + m) * N1 + v) * blockDim.x + threadIdx.x) * kSlot; };
        auto fetch = [&](int64_t row) {
#pragma unroll
            for (int v = 0; v < N1; ++v) {
                const int64_t c = col0 + v * step, n = a.cols - c;
                x[v] = load16<WIDE>(a.x + row * a.ldx + c, n, sx);
                r[v] = a.res ? load16<WIDE>(a.res + row * a.ldr + c, n, sr) : zero;
            }
        };
        auto ahead = [&](int64_t row, int at) {
            if (row < a.rows) {
#pragma unroll
                for (int v = 0; v < N1; ++v) {
                    const int64_t c = col0 + v * step, n = a.cols - c;
                    fetch16(slot(at, 0, v), a.x + row * a.ldx + c, n, sx);
                    if (a.res) fetch16(slot(at, 1, v), a.res + row * a.ldr + c, n, sr);
                }
            }
            async_commit();
        };
        // unless WIDE, only the first row comes without the slots (512 x 999: 5.3 us, 6.5 through them)
        if constexpr (!WIDE) ahead(blockIdx.x + (int64_t)gridDim.x, 1);
        fetch(blockIdx.x);
#pragma unroll
        for (int v = 0; v < N1; ++v) w[v] = load16<WIDE>(a.weight + col0 + v * step, a.cols - col0 - v * step, sw);
        for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
            if (!WIDE && row != blockIdx.x) {
                async_wait_older();
#pragma unroll
                for (int v = 0; v < N1; ++v) {
                    const int64_t c = col0 + v * step, n = a.cols - c;
                    x[v] = take16(slot(turn, 0, v), a.x + row * a.ldx + c, n);
                    r[v] = a.res ? take16(slot(turn, 1, v), a.res + row * a.ldr + c, n) : zero;
                }
            }
            float2 t[N1][8];
            float sq = 0.f;
#pragma unroll
            for (int v = 0; v < N1; ++v) {
                sums(x[v], r[v], t[v]);
                sq += squares(t[v]);
            }
            if (WIDE && row + gridDim.x < a.rows) fetch(row + gridDim.x);
            const float2 sum = block_sum2(sq, sh[turn]);
            if constexpr (!WIDE) ahead(row + 2 * (int64_t)gridDim.x, turn);      // sq has taken all that the slots held
            const float2 root = inverse_root(sum, (float)a.cols, a.inv_cols, a.eps);
#pragma unroll
            for (int v = 0; v < N1; ++v)
                if (v * step < a.cols) write(row, col0 + v * step, t[v], root, w[v]);
            if (a.rstd && threadIdx.x == 0) a.rstd[row] = root.x;
        }
    } else {
        for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
            float2 t[8];
            auto sum_at = [&](int64_t c) {
                const V16 x = load16<WIDE>(a.x + row * a.ldx + c, a.cols - c, sx);
                sums(x, a.res ? load16<WIDE>(a.res + row * a.ldr + c, a.cols - c, sr) : zero, t);
            };
            float sq = 0.f;
            for (int64_t c = col0; c - col0 < a.cols; c += step) {
                sum_at(c);
                sq += squares(t);
            }
            const float2 root = inverse_root(block_sum2(sq, sh[turn]), (float)a.cols, a.inv_cols, a.eps);
            for (int64_t c = col0; c - col0 < a.cols; c += step) {
                sum_at(c);
                write(row, c, t, root, load16<WIDE>(a.weight + c, a.cols - c, sw));
            }
            if (a.rstd && threadIdx.x == 0) a.rstd[row] = root.x;
        }
    }
}

// ------------------------------------------------------------------ norm, backward

struct NormBackArgs {
    const uint16_t *dy, *s, *weight, *ds;
    Q8 s_q8;
    const float* rstd;
    uint16_t* dx;
    float* partials;
    int64_t pitch;           // floats between rows of partials: cols, or that rounded up to a multiple of 16
    int64_t lddy, lds, ldds, lddx, rows, cols;
    int threads;             // of a group
    int parts;               // rows of partials written: the grid
    unsigned int* error;
    long long wait_limit;
};

// The CTA's threads are groups of `threads`, a row each at a time; a group takes every (groups of the grid)th row
// and keeps its part of dw: a thread owns its 16 columns in every row, in registers (HELD), the loads of the next
// row, or the next four (RING), being under way while a row is reduced and written.  Narrow rows are GROUPED: several
// rows at a time in a CTA, the groups' parts added in shared memory, so that they fill the SM without more rows of
// partials (999 x 2047: 14.3 us with a group per CTA, 10 with four).  Rows wider than 512 threads hold are read
// twice (from L2), dw's part in the CTA's row of `partials`.
template <bool HELD, bool WIDE, bool GROUPED, bool KEPT8, bool RING>
__global__ void __launch_bounds__(512) k_rmsnorm_backward(const __grid_constant__ NormBackArgs a) {
    __shared__ float sums[16][2][16];            // per group and turn
    extern __shared__ __align__(16) float parts_sh[];    // [group][columns of its threads]; the RING's stages or the slots
    dependent_launch_prologue();
    const int groups = GROUPED ? blockDim.x / a.threads : 1, group = GROUPED ? threadIdx.x / a.threads : 0;
    const int threads = GROUPED ? a.threads : blockDim.x, tid = threadIdx.x - group * threads;
    const int64_t step = (int64_t)threads * 16, col0 = (int64_t)tid * 16;
    const int64_t row0 = (int64_t)blockIdx.x * groups + group, stride = (int64_t)gridDim.x * groups;
    float (*sh)[16] = sums[group];
    const Span sy = span_of(a.dy, a.lddy, a.rows, a.cols), ss = span_of(a.s, a.lds, a.rows, a.cols);
    const Span sd = span_of(a.ds, a.ldds, a.rows, a.cols), sw = span_of(a.weight, 0, 1, a.cols);
    struct Row {
        V16 dy, s, ds;           // s: bf16 words, or 16 codes and their scale byte in s.w[0 .. 4]
    };
    auto fetch = [&](int64_t row, int64_t c, Row& v) {
        const int64_t n = a.cols - c;
        v.dy = load16<WIDE>(a.dy + row * a.lddy + c, n, sy);
        if constexpr (KEPT8) {
            const uint4 w = load_codes(a.s_q8.codes + row * a.s_q8.ld + c, n < 0 ? 0 : n > 16 ? 16 : (int)n);
            v.s.w[0] = w.x; v.s.w[1] = w.y; v.s.w[2] = w.z; v.s.w[3] = w.w;
            v.s.w[4] = n > 0 ? a.s_q8.scales[row * a.s_q8.lds + (c >> 7)] : 0;
        } else {
            v.s = load16<WIDE>(a.s + row * a.lds + c, n, ss);
        }
        if (a.ds) v.ds = load16<WIDE>(a.ds + row * a.ldds + c, n, sd);
    };
    // the normalised sum
    auto normalised = [&](const Row& v, float r, float2 (&xh)[8]) {
        if constexpr (KEPT8) {
            const float e = q8_scale(v.s.w[4]);
#pragma unroll
            for (int i = 0; i < 8; ++i) xh[i] = q8_mul2(q8_mul2(q8_unpack2(v.s.w[i >> 1] >> ((i & 1) * 16)), make_float2(e, e)), make_float2(r, r));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) xh[i] = q8_mul2(pair_of(v.s.w[i]), make_float2(r, r));
        }
    };
    auto dot = [](const Row& v, const V16& w, const float2 (&xh)[8]) {
        float2 d = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) d = q8_fma2(q8_mul2(pair_of(v.dy.w[i]), pair_of(w.w[i])), xh[i], d);
        return d.x + d.y;
    };
    auto write = [&](int64_t row, int64_t c, float r, float along, const Row& v, const V16& w, const float2 (&xh)[8]) {
        V16 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 g = q8_mul2(pair_of(v.dy.w[i]), pair_of(w.w[i]));
            float2 x = q8_fma2(xh[i], make_float2(-along, -along), g);
            x = a.ds ? q8_fma2(x, make_float2(r, r), pair_of(v.ds.w[i])) : q8_mul2(x, make_float2(r, r));
            o.w[i] = pack_bf16x2(x.x, x.y);
        }
        store16<WIDE>(a.dx + row * a.lddx + c, o, a.cols - c);
    };
    const float inv_cols = 1.f / (float)a.cols;
    float* part = a.partials + (int64_t)blockIdx.x * a.pitch;
    int turn = 0;
    if constexpr (HELD) {
        Row next = {};
        float2 dw[8];
        float r_next = 0.f;
        const V16 w = load16<WIDE>(a.weight + col0, a.cols - col0, sw);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] = make_float2(0.f, 0.f);

        // RING, with one group: the CTA's rows in stages of dy, s (or its codes) and ds; thread 0 issues the copies.
        __shared__ uint64_t full[kRowStages];
        __shared__ int gave_up[2];
        const uint32_t bytes = (uint32_t)a.cols * 2, kept = KEPT8 ? bytes / 2 : bytes, stage = bytes + kept + (a.ds ? bytes : 0);
        uint8_t* ring = reinterpret_cast<uint8_t*>(parts_sh);
        const bool in = col0 < a.cols;
        auto copy = [&](int64_t row, int at) {
            uint8_t* to = ring + at * stage;
            mbar_expect_tx(full + at, stage);
            bulk_row(to, a.dy + row * a.lddy, bytes, full + at);
            bulk_row(to + bytes, KEPT8 ? (const void*)(a.s_q8.codes + row * a.s_q8.ld) : (const void*)(a.s + row * a.lds), kept, full + at);
            if (a.ds) bulk_row(to + bytes + kept, a.ds + row * a.ldds, bytes, full + at);
        };
        // Unless WIDE: [stage][dy, s, ds][thread]
        constexpr int kKept = KEPT8 ? 16 : kSlot, kSlots = 2 * kSlot + kKept;
        uint8_t* slots = reinterpret_cast<uint8_t*>(parts_sh) + (GROUPED ? blockDim.x * 64 : 0);
        auto slot = [&](int st, int before, int size) { return slots + (st * kSlots + before) * (int)blockDim.x + (int)threadIdx.x * size; };
        auto ahead = [&](int64_t row, int st) {
            const int64_t n = a.cols - col0;
            if (row < a.rows) {
                fetch16(slot(st, 0, kSlot), a.dy + row * a.lddy + col0, n, sy);
                if constexpr (!KEPT8) fetch16(slot(st, 2 * kSlot, kKept), a.s + row * a.lds + col0, n, ss);
                else if (n > 0) async16(slot(st, 2 * kSlot, kKept), a.s_q8.codes + row * a.s_q8.ld + col0, n < 16 ? (int)n : 16);
                if (a.ds) fetch16(slot(st, kSlot, kSlot), a.ds + row * a.ldds + col0, n, sd);
            }
            async_commit();
        };
        if constexpr (!WIDE) {
            ahead(row0, 0);
            ahead(row0 + stride, 1);
        }
        auto begin = [&](int64_t row) {          // what a row's turn needs besides its stage or slots, or all of the row
            r_next = a.rstd[row];
            if constexpr (WIDE && !RING) fetch(row, col0, next);
            else if (KEPT8 && in) next.s.w[4] = a.s_q8.scales[row * a.s_q8.lds + (col0 >> 7)];
        };
        if constexpr (RING) {
            if (tid == 0) {
                for (int i = 0; i < kRowStages; ++i) mbar_init(full + i, 1);
                gave_up[0] = gave_up[1] = 0;
                asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            }
            __syncthreads();
            if (tid == 0) {
#pragma unroll 1                                 // unrolled, 16384 x 4096 took 85 us instead of 76
                for (int i = 0; i < kRowStages && row0 + i * stride < a.rows; ++i) copy(row0 + i * stride, i);
                // a limit of 0: the look is here, before the loop, where it costs 6 of 83 us
                if (a.wait_limit == 0) gave_up[0] = !mbar_wait_or_look(full, 0, 0);
            }
        }
        if (row0 < a.rows) begin(row0);
        int at = 0;
        uint32_t parity = 0;
        for (int64_t row = row0; row < a.rows; row += stride, turn ^= 1) {
            if constexpr (RING) {
                if (!mbar_wait(full + at, parity, a.wait_limit)) gave_up[turn] = 1;
                const uint8_t* from = ring + at * stage;
                if (in) {
                    next.dy = row16(from + col0 * 2);
                    if constexpr (KEPT8) {
                        const uint4 q = *reinterpret_cast<const uint4*>(from + bytes + col0);
                        next.s.w[0] = q.x, next.s.w[1] = q.y, next.s.w[2] = q.z, next.s.w[3] = q.w;
                    } else {
                        next.s = row16(from + bytes + col0 * 2);
                    }
                    if (a.ds) next.ds = row16(from + bytes + kept + col0 * 2);
                }
            }
            if constexpr (!WIDE) {
                async_wait_older();
                const int64_t n = a.cols - col0;
                next.dy = take16(slot(turn, 0, kSlot), a.dy + row * a.lddy + col0, n);
                if constexpr (KEPT8) {
                    const uint4 q = *reinterpret_cast<const uint4*>(slot(turn, 2 * kSlot, kKept));
                    next.s.w[0] = in ? q.x : 0, next.s.w[1] = in ? q.y : 0, next.s.w[2] = in ? q.z : 0, next.s.w[3] = in ? q.w : 0;
                } else {
                    next.s = take16(slot(turn, 2 * kSlot, kKept), a.s + row * a.lds + col0, n);
                }
                if (a.ds) next.ds = take16(slot(turn, kSlot, kSlot), a.ds + row * a.ldds + col0, n);
            }
            const Row now = next;
            float2 xh[8];
            const float r = r_next;
            normalised(now, r, xh);
            const float d = dot(now, w, xh);
            if (row + stride < a.rows) begin(row + stride);
            const float along = group_sum(d, sh[turn], threads, group + 1) * inv_cols;
            if constexpr (!WIDE) {
                if (threads == 32) __syncwarp();
                ahead(row + 2 * stride, turn);
            }
            if constexpr (RING) {
                // the whole CTA has read the stage, and knows who gave up (the next row's flag is another)
                if (gave_up[turn]) {
                    if (tid == 0) drain_rows(full, at, parity, (a.rows - row + stride - 1) / stride, a.error);
                    break;
                }
                if (tid == 0 && row + kRowStages * stride < a.rows) copy(row + kRowStages * stride, at);
                if (++at == kRowStages) {
                    at = 0;
                    parity ^= 1;
                }
            }
            write(row, col0, r, along, now, w, xh);
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[i] = q8_fma2(pair_of(now.dy.w[i]), xh[i], dw[i]);
        }
        if constexpr (GROUPED) {                 // the groups' parts, in order
            float* mine = parts_sh + (int64_t)group * step + col0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(mine + k * 4) = make_float4(dw[2 * k].x, dw[2 * k].y, dw[2 * k + 1].x, dw[2 * k + 1].y);
            __syncthreads();
            for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
                float all = parts_sh[c];
                for (int g = 1; g < groups; ++g) all += parts_sh[g * step + c];
                part[c] = all;
            }
        } else if (col0 < a.cols) {
            if ((a.pitch & 15) == 0) {           // room for the last vector's columns past cols
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<float4*>(part + col0 + k * 4) = make_float4(dw[2 * k].x, dw[2 * k].y, dw[2 * k + 1].x, dw[2 * k + 1].y);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (col0 + i < a.cols) part[col0 + i] = (i & 1) ? dw[i >> 1].y : dw[i >> 1].x;
            }
        }
    } else {
        bool first = true;
        for (int64_t row = row0; row < a.rows; row += stride, turn ^= 1, first = false) {
            const float r = a.rstd[row];
            float d = 0.f;
            Row v;
            float2 xh[8];
            for (int64_t c = col0; c - col0 < a.cols; c += step) {
                fetch(row, c, v);
                normalised(v, r, xh);
                d += dot(v, load16<WIDE>(a.weight + c, a.cols - c, sw), xh);
            }
            const float along = group_sum(d, sh[turn], threads, group + 1) * inv_cols;
            for (int64_t c = col0; c - col0 < a.cols; c += step) {
                fetch(row, c, v);
                normalised(v, r, xh);
                write(row, c, r, along, v, load16<WIDE>(a.weight + c, a.cols - c, sw), xh);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 d = pair_of(v.dy.w[i >> 1]);
                    if (c + i < a.cols)
                        part[c + i] = (i & 1) ? fmaf(d.y, xh[i >> 1].y, first ? 0.f : part[c + i]) : fmaf(d.x, xh[i >> 1].x, first ? 0.f : part[c + i]);
                }
            }
        }
    }
}

// dw from the partial sums: a CTA takes 16 columns, 64 groups of four threads a share of the partials each,
// added in index order within a group and then over the groups.
__global__ void __launch_bounds__(256) k_rmsnorm_dw(const float* partials, int64_t count, int64_t pitch, int64_t cols,
                                                    uint16_t* dw, float scale, int first) {
    __shared__ float sh[64][17];
    dependent_launch_prologue();
    const int lane = threadIdx.x & 3, group = threadIdx.x >> 2;
    const int64_t c = (int64_t)blockIdx.x * 16 + lane * 4;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if ((pitch & 15) == 0) {                     // whole vectors: a row of partials has room past cols
#pragma unroll 8
        for (int64_t k = group; k < count; k += 64) {
            const float4 x = *reinterpret_cast<const float4*>(partials + k * pitch + c);
            sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
        }
    } else {
        for (int64_t k = group; k < count; k += 64) {
            const float* x = partials + k * pitch + c;
            sum = make_float4(sum.x + (c < cols ? x[0] : 0.f), sum.y + (c + 1 < cols ? x[1] : 0.f),
                              sum.z + (c + 2 < cols ? x[2] : 0.f), sum.w + (c + 3 < cols ? x[3] : 0.f));
        }
    }
    sh[group][lane * 4] = sum.x;
    sh[group][lane * 4 + 1] = sum.y;
    sh[group][lane * 4 + 2] = sum.z;
    sh[group][lane * 4 + 3] = sum.w;
    __syncthreads();
    // 16 threads per column add four groups each, then the 16 partial sums in a fixed tree
    const int col = threadIdx.x >> 4, part = threadIdx.x & 15;
    float all = (sh[part * 4][col] + sh[part * 4 + 1][col]) + (sh[part * 4 + 2][col] + sh[part * 4 + 3][col]);
#pragma unroll
    for (int k = 1; k < 16; k <<= 1) all += __shfl_xor_sync(~0u, all, k);
    const int64_t at = (int64_t)blockIdx.x * 16 + col;
    if (part == 0 && at < cols) {
        all *= scale;
        if (!first) all += bf16_to_f32(dw[at]);
        dw[at] = f32_to_bf16(all);
    }
}

// ------------------------------------------------------------------ gated activation

struct GateArgs {
    const uint16_t *gate, *up;
    int64_t ldg, ldu, rows, cols;
    Q8 h, gate_q, up_q;
};

constexpr int kGateMost = 128;       // threads of a CTA

// A CTA takes a piece of a row, 16 columns per thread.
template <bool WIDE>
__global__ void __launch_bounds__(kGateMost) k_swiglu_q8(const __grid_constant__ GateArgs a) {
    dependent_launch_prologue();
    const int64_t row = blockIdx.x, c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 16, n = a.cols - c;
    const V16 wg = load16<WIDE>(a.gate + row * a.ldg + c, n, span_of(a.gate, a.ldg, a.rows, a.cols));
    const V16 wu = load16<WIDE>(a.up + row * a.ldu + c, n, span_of(a.up, a.ldu, a.rows, a.cols));
    float2 g[8], u[8], h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        g[i] = pair_of(wg.w[i]);
        u[i] = pair_of(wu.w[i]);
        h[i] = q8_mul2(q8_mul2(g[i], q8_sigmoid2(g[i])), u[i]);
    }
    encode16(h, n, a.h, row, c);
    if (a.gate_q.codes) encode16(g, n, a.gate_q, row, c);
    if (a.up_q.codes) encode16(u, n, a.up_q, row, c);
}

// Threads and register vectors (of 16 columns, `least` to `most` of them) for a row of `cols` columns: the fewest
// vectors per thread that keep the CTA within 512 threads; nv = 0 when the row does not fit in registers.
void row_shape(int64_t cols, int least, int most, int* threads, int* nv) {
    const int64_t vecs = (cols + 15) / 16;
    for (int k = least; k <= most; ++k) {
        const int64_t need = ((vecs + k - 1) / k + 31) / 32 * 32;
        if (need <= 512) {
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
    // As many CTAs as are resident: 640 threads per SM, or 512 with two vectors in their registers.  One vector per
    // thread, except where its CTAs of 256 threads and more fill 512 threads of an SM only and not all rows are
    // resident at once: then two, which share what a thread does once per row (16384 x 4096: 93 us with two, 109 with
    // one; 16384 x 2560: 77 and 61; 300 x 4096: 4.4 and 3.3; 4096 x 512: 6.5 and 5.9).
    const int sms = q8_host::sm_count();
    auto ctas = [&] { return sms * std::max(1, (nv == 2 ? 512 : 640) / threads); };
    row_shape(a.cols, 1, 2, &threads, &nv);
    if (nv == 1 && threads >= 256 && a.rows > ctas()) row_shape(a.cols, 2, 2, &threads, &nv);
    const int64_t room = ctas();
    const dim3 grid((unsigned)(a.rows < room ? a.rows : room)), block(threads);
    const size_t smem = WIDE ? 0 : (size_t)kSlotStages * 2 * nv * threads * kSlot;
    static std::atomic<uint64_t> ready[2];
    if (!WIDE && nv > 0) {
        const cudaError_t e = ready_once(ready[nv - 1], nv == 1 ? (const void*)k_rmsnorm_q8<1, WIDE> : (const void*)k_rmsnorm_q8<2, WIDE>,
                                         kSlotStages * 2 * 512 * kSlot * nv);
        if (e != cudaSuccess) return e;
    }
    switch (nv) {
        case 1: return launch_kernel(k_rmsnorm_q8<1, WIDE>, grid, block, smem, st, a);
        case 2: return launch_kernel(k_rmsnorm_q8<2, WIDE>, grid, block, smem, st, a);
        default: return launch_kernel(k_rmsnorm_q8<0, WIDE>, grid, block, 0, st, a);
    }
}

// Narrow rows: groups of threads in CTAs of about 512, one per SM.  Rows of 256 threads and more: a CTA each, as many
// as are resident (16384 x 4096 in groups of two took 98 us instead of 87-90; 512 x 8192 with two CTAs of 512 threads
// to an SM, which take turns, 15.3 instead of 11.5).
template <bool WIDE, bool KEPT8>
cudaError_t launch_norm_back(NormBackArgs& a, int64_t parts, cudaStream_t st) {
    int nv;
    row_shape(a.cols, 1, 1, &a.threads, &nv);             // two vectors, dw's sums and the inputs do not fit in registers
    const int groups = nv == 1 && a.threads < 256 ? 512 / a.threads : 1;
    // a row read twice: more CTAs than are resident, which even out (4096 x 9000: 505 us, 528 with one per SM)
    const int per_sm = groups > 1 || (nv == 1 && a.threads > 256) ? 1 : 2;
    const int64_t room = per_sm * (int64_t)q8_host::sm_count(), need = (a.rows + groups - 1) / groups;
    parts = parts < room ? parts : room;
    a.parts = (int)(parts < need ? parts : need);
    const dim3 grid((unsigned)a.parts), block(groups * a.threads);
    // Rows of a CTA each, of a multiple of 16 columns, aligned, and many per CTA: through a ring in shared memory.
    // Registers hold no more than the next row, too few bytes in flight (16384 x 4096 with kept codes: 76 us, and 85
    // without the ring; 16384 x 8192: 154 and 180).  With 13 rows per CTA both take the same time, with fewer and with
    // groups the ring is up to 10 % slower.
    if constexpr (WIDE) {
        if (nv == 1 && groups == 1 && (a.cols & 15) == 0 && a.rows >= 16 * (int64_t)a.parts) {
            static std::atomic<uint64_t> ready{0};
            const size_t smem = kRowStages * (size_t)a.cols * ((KEPT8 ? 3 : 4) + (a.ds ? 2 : 0));
            cudaError_t e = error_word(&a.error);
            a.wait_limit = wait_limit().load(std::memory_order_relaxed);
            if (e == cudaSuccess) e = ready_once(ready, (const void*)k_rmsnorm_backward<true, true, false, KEPT8, true>, kRowSmem);
            if (e != cudaSuccess) return e;
            return launch_kernel(k_rmsnorm_backward<true, true, false, KEPT8, true>, grid, block, smem, st, a);
        }
    }
    const size_t smem = (groups > 1 ? groups * a.threads * 64 : 0) +
                        (WIDE ? 0 : (size_t)kSlotStages * groups * a.threads * (2 * kSlot + (KEPT8 ? 16 : kSlot)));
    if (nv == 1) {
        auto* kern = groups > 1 ? k_rmsnorm_backward<true, WIDE, true, KEPT8, false> : k_rmsnorm_backward<true, WIDE, false, KEPT8, false>;
        static std::atomic<uint64_t> ready[2];
        const cudaError_t e = ready_once(ready[groups > 1], (const void*)kern, 512 * (64 + kSlotStages * 3 * kSlot));
        if (e != cudaSuccess) return e;
        return launch_kernel(kern, grid, block, smem, st, a);
    }
    return launch_kernel(k_rmsnorm_backward<false, WIDE, false, KEPT8, false>, grid, block, 0, st, a);
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
    a.inv_cols = 1.f / (float)cols;
    a.s = (uint16_t*)s;
    a.rstd = rstd;
    const bool w = wide(x, ldx, 32) && (!residual || wide(residual, ldr, 32)) && wide(weight, 0, 32) && (!s || wide(s, lds, 32));
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
    const bool w = wide(dy, lddy, 32) && (!s || wide(s, lds, 32)) && wide(weight, 0, 32) && (!ds || wide(ds, ldds, 32)) && wide(dx, lddx, 32);
    const cudaStream_t st = (cudaStream_t)stream;
    // rows of partial sums start at multiples of 16 floats where the scratch holds one such row, so an odd width
    // uses a few rows of scratch less
    a.pitch = (cols + 15) / 16 * 16;
    if (n_partials > int64_t(1) << 30) n_partials = int64_t(1) << 30;
    if (n_partials * cols < a.pitch) a.pitch = cols;
    int64_t parts = n_partials * cols / a.pitch;
    if (parts > ZS_Q8_MAX_PARTIALS) parts = ZS_Q8_MAX_PARTIALS;
    if (rows > 0) {
        const cudaError_t e = s_q8 ? (w ? zs::launch_norm_back<true, true>(a, parts, st) : zs::launch_norm_back<false, true>(a, parts, st))
                                   : (w ? zs::launch_norm_back<true, false>(a, parts, st) : zs::launch_norm_back<false, false>(a, parts, st));
        ZS_Q8_TRY(cuda_status(fn, e));
    }
    return cuda_status(fn, zs::launch_kernel(zs::k_rmsnorm_dw, dim3((unsigned)((cols + 15) / 16)), dim3(256), 0, st,
                                             (const float*)partials, (int64_t)a.parts, a.pitch, cols, (uint16_t*)dw, scale, (int)first));
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
    // the CTA size of 64, 96 or 128 whose pieces leave the fewest threads without columns (larger CTAs leave the SM
    // less full: 148 us instead of 118 at 8192 x 11008 with 352 threads)
    const int64_t vecs = (cols + 15) / 16;
    int threads = zs::kGateMost;
    for (int t = 96; t >= 64; t -= 32)
        if ((vecs + t - 1) / t * t < (vecs + threads - 1) / threads * threads) threads = t;
    const bool w = wide(gate, ldg, 32) && wide(up, ldu, 32);
    const cudaStream_t st = (cudaStream_t)stream;
    // as many columns at a time as a launch has pieces for: a column range that starts at a block is a matrix itself
    const int64_t most = int64_t(65535) * threads * 16;
    for (int64_t left = cols; left > 0; left -= most) {
        a.cols = left < most ? left : most;
        const dim3 grid((unsigned)rows, (unsigned)((a.cols + 16 * threads - 1) / (16 * threads))), block(threads);
        ZS_Q8_TRY(cuda_status(fn, w ? zs::launch_kernel(zs::k_swiglu_q8<true>, grid, block, 0, st, a)
                                    : zs::launch_kernel(zs::k_swiglu_q8<false>, grid, block, 0, st, a)));
        a.gate += most;
        a.up += most;
        for (zs::Q8* q : {&a.h, &a.gate_q, &a.up_q}) {
            if (!q->codes) continue;
            q->codes += most;
            q->scales += most / ZS_Q8_BLOCK;
        }
    }
    return ZS_OK;
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
