// AdamW over many tensors at once, and the norm of their gradients (include/zs.h, "many tensors at once").
//
// A launch carries the table of up to kTableMost tensors in its parameters (no device memory, nothing to upload, and a
// captured launch keeps it), and its warps take blocks of 256 elements in turn, whatever tensor they belong to.  All of it
// moves bytes: with bf16 gradients 28 per element and states of 32 bits, 16.06 with states of 8 bits.
#include <cmath>
#include <cstring>

#include "q8.cuh"

namespace zs {

namespace {

constexpr int kBlock = ZS_STATE_BLOCK;
static_assert(kBlock == 256, "a warp's block: eight elements per lane");
constexpr int kTableMost = 448, kTableFew = 48;      // a launch's parameters are at most 32764 bytes; few tensors: under 4 KB
constexpr int64_t kAligned = int64_t(1) << 62, kNoDecay = int64_t(1) << 61, kCount = kNoDecay - 1;

struct Entry {
    const void* grad;
    float* master;
    uint16_t* param;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;                       // elements, kAligned, kNoDecay
};

template <int CAP>
struct Table {
    Entry t[CAP];
    uint32_t first[CAP];             // blocks of the tensors before
    uint32_t key[CAP];               // of the tensor's random bits
    uint32_t blocks;
    int count;
    AdamScalars s;
    float inv_root;                  // 1 / s.sqrt_bc2
    const float* factor;
    float* partials;
    int add;                         // the norm's partial sums: what earlier launches left counts too
};
static_assert(sizeof(Table<kTableMost>) <= 32764 && sizeof(Table<kTableFew>) <= 4096, "a launch's parameters");

// The tensor that block u belongs to; u >= first[at].
template <int CAP>
__device__ __forceinline__ int find(const Table<CAP>& a, uint32_t u, int at) {
    int past = a.count;
    while (past - at > 1) {
        const int mid = (at + past) >> 1;
        if (a.first[mid] <= u) at = mid;
        else past = mid;
    }
    return at;
}

// ------------------------------------------------------------------ eight values per lane

// A lane's values of a block: neighbours (8 * lane + j) where the block is whole and every array aligned, else
// 32 * j + lane, so that unaligned arrays too are read and written line by line.
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "l"(p));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]),
                 "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
}

template <bool G32>
__device__ __forceinline__ void load_grad8(const void* grad, int64_t at, float (&g)[8]) {
    if (G32) {
        load8(static_cast<const float*>(grad) + at, g);
    } else {
        const BfVec<8> v = ld_bf<8>(static_cast<const uint16_t*>(grad) + at);
        unpack(v, g);
    }
}
template <bool G32>
__device__ __forceinline__ float load_grad(const void* grad, int64_t at) {
    return G32 ? __ldcs(static_cast<const float*>(grad) + at) : bf16_to_f32(__ldcs(static_cast<const uint16_t*>(grad) + at));
}

// ------------------------------------------------------------------ states in 8 bits

// The finalizer of murmur3's 32-bit hash (A. Appleby): every bit of x changes every bit of the result about half the time.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x85ebca6bu;
    x = (x ^ (x >> 13)) * 0xc2b2ae35u;
    return x ^ (x >> 16);
}

// e4m3 code of |t| <= 448 (and rounding), up or down by 16 random bits.  Times 2^-120 the code's bits are fp32's from bit
// 20 on, subnormal codes among them, and what lies below is the distance from the lower code.
__device__ __forceinline__ uint32_t state_code(float t, uint32_t random16) {
    const uint32_t c = (__float_as_uint(fabsf(t) * 0x1p-120f) + (random16 << 4)) >> 20;
    return c < 0x7e ? c : 0x7e;
}

constexpr float kLeastTop = 0x1p-100f;       // blocks below are zeros: 448 / top would pass fp32's range

// A block's scale and what its values are multiplied by; top: the largest magnitude in the warp, as bits.
__device__ __forceinline__ float block_scale(uint32_t top, float& inverse) {
    const float t = __uint_as_float(top);
    const bool some = t >= kLeastTop;
    inverse = some ? __fdividef(448.f, t) : 0.f;
    return some ? t * (1.f / 448.f) : 0.f;
}

// The values x in 8 bits, POSITIVE: they are not negative, and what is above 0 gets no code 0.  `random`: 16 bits per
// value, the lower or the upper half.  Infinities and NaN have the code NaN and leave the scale alone.
template <bool POSITIVE>
__device__ __forceinline__ void encode_state(const float (&x)[8], const uint32_t (&random)[8], uint32_t (&code)[8], float& scale) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
    top = __reduce_max_sync(~0u, top);
    const bool bad = top >= 0x7f800000u;
    if (bad) {
        top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(x[j]) & 0x7fffffffu;
            if (b < 0x7f800000u) top = max(top, b);
        }
        top = __reduce_max_sync(~0u, top);
    }
    float inverse;
    scale = block_scale(top, inverse);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = x[j] * inverse;
        uint32_t c = state_code(t, POSITIVE ? random[j] >> 16 : random[j] & 0xffffu);
        if (POSITIVE) c = c == 0 && t > 0.f ? 1 : c;
        if (!POSITIVE) c |= (__float_as_uint(t) >> 24) & 0x80u;
        if (bad && (__float_as_uint(x[j]) & 0x7fffffffu) >= 0x7f800000u) c = 0x7f;
        code[j] = c;
    }
}

__device__ __forceinline__ uint2 pack_codes(const uint32_t (&c)[8]) {
    return make_uint2(c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24), c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24));
}
__device__ __forceinline__ float code_value(uint32_t c) { return q8_unpack2(c).x; }

// ------------------------------------------------------------------ the step

// One block of a tensor per warp.
template <bool G32, bool Q, int CAP>
__global__ void __launch_bounds__(256) k_adamw_tensors(const __grid_constant__ Table<CAP> a) {
    dependent_launch_prologue();
    const int lane = threadIdx.x & 31;
    const uint32_t warps = (uint32_t)(gstride() >> 5);
    const float factor = a.factor ? *a.factor : 1.f;
    if (isnan(factor)) return;                   // gradients that are not finite: no step
    int e = 0;
    for (uint32_t u = (uint32_t)(gtid() >> 5); u < a.blocks; u += warps) {
        e = find(a, u, e);
        const Entry& t = a.t[e];
        const int64_t n = t.n & kCount, block = u - a.first[e], begin = block * kBlock;
        const bool whole = (t.n & kAligned) && n - begin >= kBlock;
        const int64_t at = begin + (whole ? lane * 8 : lane);
        float g[8], p[8], m[8], v[8];
        float ms = 0.f, vs = 0.f;
        if (Q) {
            ms = t.m_scale[block];
            vs = t.v_scale[block];
        }
        if (whole) {
            load_grad8<G32>(t.grad, at, g);
            load8(t.master + at, p);
            if (Q) {
                const uint2 cm = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + at));
                const uint2 cv = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + at));
                q8_unpack4(cm.x, ms, m);
                q8_unpack4(cm.y, ms, m + 4);
                q8_unpack4(cv.x, vs, v);
                q8_unpack4(cv.y, vs, v + 4);
            } else {
                load8(static_cast<const float*>(t.m) + at, m);
                load8(static_cast<const float*>(t.v) + at, v);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t i = at + 32 * j;
                const bool live = i < n;
                g[j] = live ? load_grad<G32>(t.grad, i) : 0.f;
                p[j] = live ? __ldcs(t.master + i) : 0.f;
                if (Q) {
                    m[j] = live ? code_value(static_cast<const uint8_t*>(t.m)[i]) * ms : 0.f;
                    v[j] = live ? code_value(static_cast<const uint8_t*>(t.v)[i]) * vs : 0.f;
                } else {
                    m[j] = live ? __ldcs(static_cast<const float*>(t.m) + i) : 0.f;
                    v[j] = live ? __ldcs(static_cast<const float*>(t.v) + i) : 0.f;
                }
            }
        }
        AdamScalars s = a.s;
        if (t.n & kNoDecay) s.decay = 1.f;
        uint32_t cm[8], cv[8];
        if (Q) {
            const uint32_t key = mix(a.key[e] + (uint32_t)(begin >> 32));
            uint32_t random[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = g[j] * factor;
                m[j] = fmaf(s.beta1, m[j], s.c1 * x);
                const float y = fmaf(s.beta2, v[j] * v[j], s.c2 * (x * x));
                asm("sqrt.approx.f32 %0, %1;" : "=f"(v[j]) : "f"(y));
                p[j] = fmaf(-s.step_size, __fdividef(m[j], fmaf(v[j], a.inv_root, s.eps)), p[j] * s.decay);
                random[j] = mix((uint32_t)(at + (whole ? j : 32 * j)) ^ key);
            }
            encode_state<false>(m, random, cm, ms);
            encode_state<true>(v, random, cv, vs);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) adamw_elem(__fmul_rn(g[j], factor), p[j], m[j], v[j], s);
        }
        if (whole) {
            store8(t.master + at, p);
            if (t.param) st_bf<8>(t.param + at, pack(p));
            if (Q) {
                __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + at), pack_codes(cm));
                __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + at), pack_codes(cv));
            } else {
                store8(static_cast<float*>(t.m) + at, m);
                store8(static_cast<float*>(t.v) + at, v);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t i = at + 32 * j;
                if (i >= n) break;
                t.master[i] = p[j];
                if (t.param) t.param[i] = f32_to_bf16(p[j]);
                if (Q) {
                    static_cast<uint8_t*>(t.m)[i] = (uint8_t)cm[j];
                    static_cast<uint8_t*>(t.v)[i] = (uint8_t)cv[j];
                } else {
                    static_cast<float*>(t.m)[i] = m[j];
                    static_cast<float*>(t.v)[i] = v[j];
                }
            }
        }
        if (Q && lane == 0) {
            t.m_scale[block] = ms;
            t.v_scale[block] = vs;
        }
    }
}

// ------------------------------------------------------------------ the gradients' norm

// Sum over the CTA's 256 threads, in thread 0.
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double sh[8];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(~0u, x, k);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < 8; ++w) x += sh[w];
    return x;
}

// A lane adds eight squares in fp32, and those sums in fp64.  The CTAs' sums are rounded to fp32 (they are as many as the
// caller has room for, each of its own blocks, so the same bits every time) and added by one CTA.
template <bool G32, int CAP>
__global__ void __launch_bounds__(256) k_grad_norm(const __grid_constant__ Table<CAP> a) {
    dependent_launch_prologue();
    const int lane = threadIdx.x & 31;
    const uint32_t warps = (uint32_t)(gstride() >> 5);
    double sum = 0.0;
    int e = 0;
    for (uint32_t u = (uint32_t)(gtid() >> 5); u < a.blocks; u += warps) {
        e = find(a, u, e);
        const Entry& t = a.t[e];
        const int64_t n = t.n & kCount, begin = (int64_t)(u - a.first[e]) * kBlock;
        const bool whole = (t.n & kAligned) && n - begin >= kBlock;
        float g[8];
        if (whole) {
            load_grad8<G32>(t.grad, begin + lane * 8, g);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t i = begin + lane + 32 * j;
                g[j] = i < n ? load_grad<G32>(t.grad, i) : 0.f;
            }
        }
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) q = fmaf(g[j], g[j], q);
        sum += q;
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) a.partials[blockIdx.x] = (float)(a.add ? sum + a.partials[blockIdx.x] : sum);
}

__global__ void __launch_bounds__(256) k_grad_norm_end(const float* partials, int n, float max_norm, float* out) {
    dependent_launch_prologue();
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += 256) sum += partials[i];
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        const float norm = (float)sqrt(sum);
        // not finite: no factor, and a step given it is not taken
        const float factor = __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f));
        out[0] = norm;
        out[1] = isfinite(norm) ? fminf(factor, 1.f) : __int_as_float(0x7fffffff);
    }
}

// ------------------------------------------------------------------ host

using q8_host::cuda_status;
using q8_host::fail;

bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

std::string of(const char* name, int i) { return std::string(name) + " of tensor " + std::to_string(i); }

int check_tensor(const char* fn, const zs_tensor& t, int i, int grad_bytes, int state_bits, bool step) {
    if (t.n < 0 || t.n > (int64_t(1) << 40)) return fail(fn, of("n", i) + " out of range");
    if (t.n == 0) return ZS_OK;
    if (!t.grad) return fail(fn, of("grad", i) + " is NULL");
    if (!aligned(t.grad, grad_bytes)) return fail(fn, of("grad", i) + " is not aligned to its elements");
    if (!step) return ZS_OK;
    if (!t.master || !t.m || !t.v) return fail(fn, of("master, m or v", i) + " is NULL");
    if (!aligned(t.master, 4) || (state_bits == 32 && (!aligned(t.m, 4) || !aligned(t.v, 4))))
        return fail(fn, of("master, m or v", i) + " is not 4-byte aligned");
    if (!aligned(t.param, 2)) return fail(fn, of("param", i) + " is not 2-byte aligned");
    if (state_bits == 8 && (!t.m_scale || !t.v_scale || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4)))
        return fail(fn, of("m_scale or v_scale", i) + " is NULL or not 4-byte aligned");
    return ZS_OK;
}

// Whether a whole block's values are read and written eight at a time.
bool wide_blocks(const zs_tensor& t, int grad_bytes, int state_bits, bool step) {
    if (!aligned(t.grad, 8 * grad_bytes)) return false;
    if (!step) return true;
    return aligned(t.master, 32) && aligned(t.param, 16) && aligned(t.m, state_bits) && aligned(t.v, state_bits);
}

// Calls launch(table, first) for the tensors, as many at a time as a launch's parameters hold.
template <int CAP, typename F>
cudaError_t by_table(const zs_tensor* tensors, int count, int grad_bytes, int state_bits, bool step, uint32_t seed, Table<CAP>& a, F launch) {
    bool first = true;
    int i = 0;
    do {
        a.count = 0;
        uint64_t blocks = 0;
        for (; i < count && a.count < CAP; ++i) {
            const zs_tensor& t = tensors[i];
            if (t.n == 0) continue;
            const uint64_t more = (uint64_t)(t.n + kBlock - 1) / kBlock;
            if (a.count && blocks + more > 0x7fffffffu) break;
            Entry& e = a.t[a.count];
            e = Entry{t.grad, t.master, (uint16_t*)t.param, t.m, t.v, t.m_scale, t.v_scale, t.n};
            if (wide_blocks(t, grad_bytes, state_bits, step)) e.n |= kAligned;
            if (t.no_decay) e.n |= kNoDecay;
            a.first[a.count] = (uint32_t)blocks;
            a.key[a.count] = mix(seed + 0x9e3779b9u * ((uint32_t)i + 1));
            blocks += more;
            ++a.count;
        }
        a.blocks = (uint32_t)blocks;
        if (a.count || first) {
            const cudaError_t rc = launch(a, first);
            if (rc != cudaSuccess) return rc;
        }
        first = false;
    } while (i < count);
    return cudaSuccess;
}

constexpr int kStepCtas = 6, kNormCtas = 8;          // resident CTAs per SM

unsigned grid_of(uint32_t blocks, int64_t most) {
    const int64_t ctas = ((int64_t)blocks + 7) / 8;
    return (unsigned)(ctas < 1 ? 1 : ctas < most ? ctas : most);
}

template <bool G32, bool Q, int CAP>
cudaError_t step_tensors(const zs_tensor* tensors, int count, uint32_t seed, Table<CAP>& a, cudaStream_t st) {
    return by_table<CAP>(tensors, count, G32 ? 4 : 2, Q ? 8 : 32, true, seed, a, [&](const Table<CAP>& t, bool) {
        if (!t.count) return cudaSuccess;
        return launch_kernel(k_adamw_tensors<G32, Q, CAP>, dim3(grid_of(t.blocks, (int64_t)q8_host::sm_count() * kStepCtas)), dim3(256), 0, st, t);
    });
}

template <int CAP>
cudaError_t step_any(const zs_tensor* tensors, int count, bool g32, bool q, uint32_t seed, const AdamScalars& s, const float* factor,
                     cudaStream_t st) {
    Table<CAP> a;
    a.s = s;
    a.inv_root = (float)(1.0 / (double)s.sqrt_bc2);
    a.factor = factor;
    return g32 ? (q ? step_tensors<true, true>(tensors, count, seed, a, st) : step_tensors<true, false>(tensors, count, seed, a, st))
               : (q ? step_tensors<false, true>(tensors, count, seed, a, st) : step_tensors<false, false>(tensors, count, seed, a, st));
}

template <bool G32, int CAP>
cudaError_t norm_tensors(const zs_tensor* tensors, int count, float* partials, int n_partials, cudaStream_t st) {
    Table<CAP> a;
    a.partials = partials;
    return by_table<CAP>(tensors, count, G32 ? 4 : 2, 32, false, 0, a, [&](Table<CAP>& t, bool first) {
        t.add = !first;
        return launch_kernel(k_grad_norm<G32, CAP>, dim3((unsigned)n_partials), dim3(256), 0, st, t);
    });
}

int check_list(const char* fn, const zs_tensor* tensors, int32_t n_tensors, int32_t grad_bytes, int32_t state_bits, bool step) {
    if (n_tensors < 0) return fail(fn, "n_tensors is negative");
    if (!tensors && n_tensors > 0) return fail(fn, "tensors is NULL");
    if (grad_bytes != 2 && grad_bytes != 4) return fail(fn, "grad_bytes must be 2 (bf16) or 4 (fp32)");
    if (step && state_bits != 8 && state_bits != 32) return fail(fn, "state_bits must be 8 or 32");
    for (int i = 0; i < n_tensors; ++i) ZS_Q8_TRY(check_tensor(fn, tensors[i], i, grad_bytes, state_bits, step));
    return ZS_OK;
}

}  // namespace

}  // namespace zs

using namespace zs::q8_host;

extern "C" int zs_adamw_tensors(const zs_tensor* tensors, int32_t n_tensors, int32_t grad_bytes, int32_t state_bits,
                                const zs_adamw_hparams* hp, int64_t step, const float* factor, uint32_t seed, void* stream) {
    static const char* fn = "zs_adamw_tensors";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    if (!hp) return fail(fn, "hparams is NULL");
    if (step < 1) return fail(fn, "step must be >= 1 (1-based)");
    for (float x : {hp->lr, hp->beta1, hp->beta2, hp->eps, hp->weight_decay})
        if (!std::isfinite(x)) return fail(fn, "hyper-parameters must be finite");
    if (!(hp->beta1 >= 0.f && hp->beta1 < 1.f && hp->beta2 >= 0.f && hp->beta2 < 1.f)) return fail(fn, "betas must lie in [0, 1)");
    if (!zs::aligned(factor, 4)) return fail(fn, "factor is not 4-byte aligned");
    ZS_Q8_TRY(zs::check_list(fn, tensors, n_tensors, grad_bytes, state_bits, true));
    float sc[8];
    ZS_Q8_TRY(zs_adamw_scalars(hp, step, sc));
    const zs::AdamScalars s{sc[0], sc[1], sc[2], sc[3], sc[4], sc[5], sc[6], sc[7]};
    const cudaStream_t st = (cudaStream_t)stream;
    return cuda_status(fn, n_tensors <= zs::kTableFew
                               ? zs::step_any<zs::kTableFew>(tensors, n_tensors, grad_bytes == 4, state_bits == 8, seed, s, factor, st)
                               : zs::step_any<zs::kTableMost>(tensors, n_tensors, grad_bytes == 4, state_bits == 8, seed, s, factor, st));
}

extern "C" int zs_grad_norm(const zs_tensor* tensors, int32_t n_tensors, int32_t grad_bytes, float max_norm, float* partials,
                            int64_t n_partials, float* out, void* stream) {
    static const char* fn = "zs_grad_norm";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    if (!(max_norm > 0.f) || !std::isfinite(max_norm)) return fail(fn, "max_norm must be positive and finite");
    if (!partials || !zs::aligned(partials, 4)) return fail(fn, "partials is NULL or not 4-byte aligned");
    if (n_partials < 1) return fail(fn, "n_partials must be at least 1");
    if (!out || !zs::aligned(out, 4)) return fail(fn, "out is NULL or not 4-byte aligned");
    ZS_Q8_TRY(zs::check_list(fn, tensors, n_tensors, grad_bytes, 32, false));
    const cudaStream_t st = (cudaStream_t)stream;
    int64_t blocks = 0;
    for (int i = 0; i < n_tensors; ++i) blocks += (tensors[i].n + zs::kBlock - 1) / zs::kBlock;
    const int64_t most = (int64_t)sm_count() * zs::kNormCtas;
    const int n = (int)zs::grid_of((uint32_t)(blocks < 0x7fffffff ? blocks : 0x7fffffff), n_partials < most ? n_partials : most);
    const bool few = n_tensors <= zs::kTableFew;
    cudaError_t e;
    if (grad_bytes == 4) e = few ? zs::norm_tensors<true, zs::kTableFew>(tensors, n_tensors, partials, n, st) : zs::norm_tensors<true, zs::kTableMost>(tensors, n_tensors, partials, n, st);
    else e = few ? zs::norm_tensors<false, zs::kTableFew>(tensors, n_tensors, partials, n, st) : zs::norm_tensors<false, zs::kTableMost>(tensors, n_tensors, partials, n, st);
    if (e == cudaSuccess) e = zs::launch_kernel(zs::k_grad_norm_end, dim3(1), dim3(256), 0, st, (const float*)partials, n, max_norm, out);
    return cuda_status(fn, e);
}
