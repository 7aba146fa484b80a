// AdamW over many tensors at once, and the norm of their gradients (include/zs.h, "many tensors at once").
//
// A launch carries the table of up to kTableMost tensors in its parameters (no device memory, nothing to upload, and a
// captured launch keeps it), and its CTAs take tiles of eight blocks of 256 elements in turn, whatever tensor they belong
// to.  All of it moves bytes: with bf16 gradients 28 per element and states of 32 bits, 16.06 with states of 8 bits.
#include <cfloat>
#include <cmath>

#include "q8_tma.cuh"

namespace zs {

namespace {

constexpr int kBlock = ZS_STATE_BLOCK;
static_assert(kBlock == 256, "a warp's block: eight elements per lane");
constexpr int kTileBlocks = 8, kTile = kTileBlocks * kBlock;         // a tile: a block for each of eight warps
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
    uint32_t first[CAP];             // tiles of the tensors before
    uint32_t key[CAP];               // of the tensor's random bits
    uint32_t tiles;
    int count;
    AdamScalars s;
    float inv_root;                  // 1 / s.sqrt_bc2
    float eps;                       // s.eps, not subnormal
    float one;                       // 1, which the compiler does not know (sum2)
    uint32_t run;                    // tiles of a CTA
    const float* factor;
    float* partials;
    float* out;                      // where one CTA has all of the norm's sum
    float max_norm;
    int add;                         // the norm's partial sums: what earlier launches left counts too
    unsigned int* error;
    long long wait_limit;
};
static_assert(sizeof(Table<kTableMost>) <= 32764 && sizeof(Table<kTableFew>) <= 4096, "a launch's parameters");

// The tensor that tile u belongs to, where an earlier tile belonged to `at`.
template <int CAP>
__device__ __forceinline__ int find(const Table<CAP>& a, uint32_t u, int at) {
    if (at + 1 >= a.count || u < a.first[at + 1]) return at;
    int past = a.count;
    while (past - at > 1) {
        const int mid = (at + past) >> 1;
        if (a.first[mid] <= u) at = mid;
        else past = mid;
    }
    return at;
}

// ------------------------------------------------------------------ eight values per lane

// A lane's values of a block: neighbours (8 * lane + j) where every array is aligned, else 32 * j + lane, so that unaligned
// arrays too are read and written line by line.
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
//
// Every operation up to a code is rounded once, in the order of the definition, so that a state's bits do not depend on
// the path that computed them.  With one instruction per operation a step takes about 80 per element, which is all that
// can be issued while its 16 bytes pass; hence two values per instruction wherever there is one, and no test per value
// for what is rare: blocks with infinities, NaN or magnitudes past kFastTop go through step_any.

// The finalizer of murmur3's 32-bit hash (A. Appleby): every bit of x changes every bit of the result about half the time.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x85ebca6bu;
    x = (x ^ (x >> 13)) * 0xc2b2ae35u;
    return x ^ (x >> 16);
}

constexpr float kLeastTop = 0x1p-100f;       // blocks below are zeros: 448 / top would pass fp32's range
constexpr float kFastTop = 0x1p14f;          // up to here 448 / top * 2^-120 is a normal number

// A block's scale and what its values are multiplied by; t: their largest magnitude.
__device__ __forceinline__ float block_scale(float t, float& inverse) {
    const bool some = t >= kLeastTop;
    inverse = some ? __fmul_rn(448.f, __frcp_rn(t)) : 0.f;
    return some ? __fmul_rn(t, 1.f / 448.f) : 0.f;
}

// An element's two lots of 16 random bits: m's, r's.
struct Random {
    uint32_t m, r;
};
__device__ __forceinline__ Random random_bits(uint32_t x) {          // x: the hash before its last step
    const uint32_t hi = x >> 16;
    return {(x ^ hi) & 0xffffu, hi};
}

// Magnitudes times 2^-120 have their e4m3 code from bit 20 on, subnormal codes among them, and below it their distance from
// that code: with 16 random bits added there (at most 2^20 - 16: a largest magnitude that rounding took a little past
// 448 does not reach the next) the code is that of the lower neighbour or of the upper.
__device__ __forceinline__ uint32_t raised(uint32_t bits, uint32_t random16) { return bits + (random16 << 4); }
// Four codes in the order of their elements: bits 20 to 26, and m's sign from bit 31 (a root has none, though root2 gives -0 for 0).
template <bool SIGN>
__device__ __forceinline__ uint32_t two_codes(uint32_t a, uint32_t b) {          // at bits 8 to 15 and 24 to 31
    const uint32_t w = __byte_perm(a, b, 0x7632);
    return ((w << 4) & 0x7fff7fffu) | (SIGN ? w & 0x80008000u : 0u);
}
template <bool SIGN>
__device__ __forceinline__ uint2 eight_codes(const uint32_t (&w)[8]) {
    return make_uint2(__byte_perm(two_codes<SIGN>(w[0], w[1]), two_codes<SIGN>(w[2], w[3]), 0x7531),
                      __byte_perm(two_codes<SIGN>(w[4], w[5]), two_codes<SIGN>(w[6], w[7]), 0x7531));
}

// a + b, each sum rounded once, in a form that is not contracted with the products that a and b are (as mul.rn.f32x2 and
// add.rn.f32x2 are, and a fused multiplication by a 1 that is known).
__device__ __forceinline__ float2 sum2(float2 a, float one, float2 b) { return q8_fma2(a, make_float2(one, one), b); }

// Square root rounded to nearest, given -2^66 y: from the hardware's reciprocal root one correction by the residual
// y - s^2, which fused multiplication gives exactly (P. Markstein, 1990).  Compared with __fsqrt_rn for every y of
// [2^-168, 2^54): equal; below, where the residual loses bits, 25 of the 2^26 values down to 2^-176 differ.
// 2^66 y has a normal root for every y > 0, and the result is exact to scale back; y = 0 gives -0.
__device__ __forceinline__ float2 root2(float2 minus) {
    float2 q;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(q.x) : "f"(fmaxf(-minus.x, 0x1p-126f)));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(q.y) : "f"(fmaxf(-minus.y, 0x1p-126f)));
    const float2 s = q8_mul2(minus, q), h = q8_mul2(q, make_float2(0.5f, 0.5f));         // s: minus the root
    return q8_mul2(q8_fma2(q8_fma2(s, s, minus), h, s), make_float2(-0x1p-33f, -0x1p-33f));
}

// max(top, |x.x|, |x.y|), NaN if one is.
__device__ __forceinline__ float top_nan(float top, float2 x) {
    float d;
    asm("{\n\t.reg .f32 a, b;\n\tabs.f32 a, %2;\n\tabs.f32 b, %3;\n\tmax.NaN.f32 %0, %1, a, b;\n\t}" : "=f"(d) : "f"(top), "f"(x.x), "f"(x.y));
    return d;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Within one unit in the last place; a root above 0 is at least 2^-75 and eps not subnormal, so nothing subnormal comes here.
__device__ __forceinline__ float reciprocal(float x) {
    float d;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
    return d;
}

constexpr float kUp = -0x1p66f;              // what the sums under roots are multiplied by

struct Scalars8 {
    float beta1, beta2, eps, decay, c1, c2, step_size, inv_root, one;
};

// A lane's eight elements.  m, v: their old codes; ms, vs: the block's scales.
struct Codes8 {
    uint2 m, v;
    float ms, vs;
};
__device__ __forceinline__ void decode8(uint2 c, float scale, float2 (&f)[4]) {
    f[0] = q8_mul2(q8_unpack2(c.x & 0xffffu), both(scale));
    f[1] = q8_mul2(q8_unpack2(c.x >> 16), both(scale));
    f[2] = q8_mul2(q8_unpack2(c.y & 0xffffu), both(scale));
    f[3] = q8_mul2(q8_unpack2(c.y >> 16), both(scale));
}

// One step of eight elements per lane, a block per warp.  g: the gradients, p: the masters, updated; hash: element 0's
// hash after its first shift, APART bits from one element's index to the next (0: neighbours, 5: 32 apart; below the
// first shift, so they may be put in after it).  Returns whether the block was one for this path; c holds the new states.
template <int APART>
__device__ __forceinline__ bool step8(const float2 (&g)[4], float2 (&p)[4], Codes8& c, uint32_t hash, float factor, const Scalars8& s) {
    float2 m[4], r[4];
    decode8(c.m, c.ms, m);
    decode8(c.v, c.vs, r);
    float top_m = 0.f, top_r = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 x = q8_mul2(g[k], both(factor));
        m[k] = sum2(q8_mul2(both(s.beta1), m[k]), s.one, q8_mul2(both(s.c1), x));
        r[k] = root2(sum2(q8_mul2(both(s.beta2 * kUp), q8_mul2(r[k], r[k])), s.one, q8_mul2(both(s.c2 * kUp), q8_mul2(x, x))));
        top_m = top_nan(top_m, m[k]);
        top_r = top_nan(top_r, r[k]);
    }
    const uint32_t bits_m = __reduce_max_sync(~0u, __float_as_uint(top_m)), bits_r = __reduce_max_sync(~0u, __float_as_uint(top_r));
    if (max(bits_m, bits_r) > __float_as_uint(kFastTop)) return false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 den = q8_fma2(r[k], both(s.inv_root), both(s.eps));
        const float2 step = q8_mul2(m[k], make_float2(reciprocal(den.x), reciprocal(den.y)));
        p[k] = q8_fma2(both(-s.step_size), step, q8_mul2(p[k], both(s.decay)));
    }
    float inv_m, inv_r;
    c.ms = block_scale(__uint_as_float(bits_m), inv_m);
    c.vs = block_scale(__uint_as_float(bits_r), inv_r);
    inv_m *= 0x1p-120f;
    inv_r *= 0x1p-120f;
    const uint32_t least = c.vs > 0.f ? 1u << 20 : 0u;
    uint32_t wm[8], wr[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 tm = q8_mul2(m[k], both(inv_m)), tr = q8_mul2(r[k], both(inv_r));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t x = (hash ^ (uint32_t)((2 * k + h) << APART)) * 0x85ebca6bu;
            x = (x ^ (x >> 13)) * 0xc2b2ae35u;
            const Random random = random_bits(x);
            wm[2 * k + h] = raised(__float_as_uint(h ? tm.y : tm.x), random.m);
            // above 0 a root's bits are above `least`
            wr[2 * k + h] = max(raised(__float_as_uint(h ? tr.y : tr.x), random.r), min(__float_as_uint(h ? r[k].y : r[k].x), least));
        }
    }
    c.m = eight_codes<true>(wm);
    c.v = eight_codes<false>(wr);
    return true;
}

// A state's values in 8 bits, whatever they are: infinities and NaN have the code NaN and leave the scale alone.
template <bool POSITIVE>
__device__ __forceinline__ uint2 encode8_any(const float (&x)[8], uint32_t hash, float& scale) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (isfinite(x[j])) top = max(top, __float_as_uint(fabsf(x[j])));
    const float most = __uint_as_float(__reduce_max_sync(~0u, top));
    float inverse;
    scale = block_scale(most, inverse);
    // one product, rounded once, as in step8 where that can be; beyond kFastTop the two factors have to stay apart
    const bool once = most <= kFastTop;
    const float by = once ? inverse * 0x1p-120f : inverse, then = once ? 1.f : 0x1p-120f;
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t h = (hash ^ (uint32_t)(32 * j)) * 0x85ebca6bu;
        h = (h ^ (h >> 13)) * 0xc2b2ae35u;
        const Random random = random_bits(h);
        uint32_t c = raised(__float_as_uint(__fmul_rn(__fmul_rn(x[j], by), then)), POSITIVE ? random.r : random.m);
        if (POSITIVE && scale > 0.f && x[j] > 0.f) c = max(c, 1u << 20);
        w[j] = isfinite(x[j]) ? c : 0x7f00000u;
    }
    return eight_codes<!POSITIVE>(w);
}
// A block of any size at any address: lane l has elements l, l + 32, .. of it, so that unaligned arrays too are read and
// written line by line.
template <bool G32>
struct Strided {
    const Entry& t;
    int64_t begin;
    int left;                        // elements of the tensor from the block on, if fewer than a block
    __device__ __forceinline__ Strided(const Entry& entry, int64_t block) : t(entry), begin(block * kBlock + (threadIdx.x & 31)) {
        const int64_t n = (entry.n & kCount) - block * kBlock;
        left = (n < kBlock ? (int)n : kBlock) - (int)(threadIdx.x & 31);
    }
    __device__ __forceinline__ bool live(int j) const { return 32 * j < left; }
    __device__ __forceinline__ void load(float (&g)[8], float (&p)[8], Codes8& c, int64_t block) const {
        uint32_t cm[8], cv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t i = begin + 32 * j;
            g[j] = live(j) ? load_grad<G32>(t.grad, i) : 0.f;
            p[j] = live(j) ? __ldcs(t.master + i) : 0.f;
            cm[j] = live(j) ? __ldcs(static_cast<const uint8_t*>(t.m) + i) : 0;
            cv[j] = live(j) ? __ldcs(static_cast<const uint8_t*>(t.v) + i) : 0;
        }
        auto pack4 = [](const uint32_t* x) { return x[0] | (x[1] << 8) | (x[2] << 16) | (x[3] << 24); };
        c = Codes8{make_uint2(pack4(cm), pack4(cm + 4)), make_uint2(pack4(cv), pack4(cv + 4)), t.m_scale[block], t.v_scale[block]};
    }
    __device__ __forceinline__ void store(const float (&p)[8], const Codes8& c, int64_t block) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!live(j)) break;
            const int64_t i = begin + 32 * j;
            t.master[i] = p[j];
            if (t.param) t.param[i] = f32_to_bf16(p[j]);
            static_cast<uint8_t*>(t.m)[i] = (uint8_t)((j < 4 ? c.m.x : c.m.y) >> (8 * (j & 3)));
            static_cast<uint8_t*>(t.v)[i] = (uint8_t)((j < 4 ? c.v.x : c.v.y) >> (8 * (j & 3)));
        }
        if ((threadIdx.x & 31) == 0) {
            t.m_scale[block] = c.ms;
            t.v_scale[block] = c.vs;
        }
    }
};

template <int CAP>
__device__ __forceinline__ Scalars8 scalars8(const Table<CAP>& a, const Entry& t) {
    return Scalars8{a.s.beta1, a.s.beta2, a.eps, t.n & kNoDecay ? 1.f : a.s.decay, a.s.c1, a.s.c2, a.s.step_size, a.inv_root, a.one};
}
// The hash of element i of a block's tensor after its first shift.
template <int CAP>
__device__ __forceinline__ uint32_t hash_of(const Table<CAP>& a, int e, int64_t i) {
    const uint32_t x = (uint32_t)i ^ mix(a.key[e] + (uint32_t)(i >> 32));
    return x ^ (x >> 16);
}

// sqrt(beta2 * rr + c2 * xx): as step8 has it, sum and root of 2^66 times as much, wherever that path has a result (sums below
// fp32's normal numbers would be rounded to other values, and so to other codes, beside a value that is not finite).
__device__ __forceinline__ float root_any(float rr, float xx, const Scalars8& s) {
    const float minus = __fadd_rn(__fmul_rn(s.beta2 * kUp, rr), __fmul_rn(s.c2 * kUp, xx));
    if (minus > -0x1p120f) return root2(make_float2(minus, minus)).x;
    return __fsqrt_rn(__fadd_rn(__fmul_rn(s.beta2, rr), __fmul_rn(s.c2, xx)));
}

// A step of a block with whatever values.
template <bool G32, int CAP>
__device__ __noinline__ void step_any(const Table<CAP>& a, int e, int64_t block, float factor) {
    const Strided<G32> at(a.t[e], block);
    const Scalars8 s = scalars8(a, a.t[e]);
    const uint32_t hash = hash_of(a, e, at.begin);
    float g[8], p[8], m[8], r[8];
    Codes8 c;
    at.load(g, p, c, block);
    q8_unpack4(c.m.x, c.ms, m);
    q8_unpack4(c.m.y, c.ms, m + 4);
    q8_unpack4(c.v.x, c.vs, r);
    q8_unpack4(c.v.y, c.vs, r + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = __fmul_rn(g[j], factor);
        m[j] = __fadd_rn(__fmul_rn(s.beta1, m[j]), __fmul_rn(s.c1, x));
        r[j] = root_any(__fmul_rn(r[j], r[j]), __fmul_rn(x, x), s);
        p[j] = fmaf(-s.step_size, __fmul_rn(m[j], reciprocal(fmaf(r[j], s.inv_root, s.eps))), __fmul_rn(p[j], s.decay));
    }
    c.m = encode8_any<false>(m, hash, c.ms);
    c.v = encode8_any<true>(r, hash, c.vs);
    at.store(p, c, block);
}

__device__ __forceinline__ void to_pairs(const float (&f)[8], float2 (&d)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = make_float2(f[2 * k], f[2 * k + 1]);
}
__device__ __forceinline__ void of_pairs(const float2 (&d)[4], float (&f)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = d[k].x;
        f[2 * k + 1] = d[k].y;
    }
}

// A step of a block that is not whole or not aligned.
template <bool G32, int CAP>
__device__ __noinline__ void step_strided(const Table<CAP>& a, int e, int64_t block, float factor) {
    const Strided<G32> at(a.t[e], block);
    float gf[8], pf[8];
    Codes8 c;
    at.load(gf, pf, c, block);
    float2 g[4], p[4];
    to_pairs(gf, g);
    to_pairs(pf, p);
    if (!step8<5>(g, p, c, hash_of(a, e, at.begin), factor, scalars8(a, a.t[e]))) {
        step_any<G32>(a, e, block, factor);
        return;
    }
    of_pairs(p, pf);
    at.store(pf, c, block);
}

// ------------------------------------------------------------------ the step

// States of 32 bits: the arithmetic of the flat step, bit for bit, for a block that is not whole or not aligned.
template <bool G32, int CAP>
__device__ __noinline__ void step_strided32(const Table<CAP>& a, int e, int64_t block, float factor) {
    const Entry& t = a.t[e];
    const int64_t n = t.n & kCount, begin = block * kBlock + (threadIdx.x & 31);
    float *tm = static_cast<float*>(t.m), *tv = static_cast<float*>(t.v);
    float g[8], p[8], m[8], v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t i = begin + 32 * j;
        const bool live = i < n;
        g[j] = live ? load_grad<G32>(t.grad, i) : 0.f;
        p[j] = live ? __ldcs(t.master + i) : 0.f;
        m[j] = live ? __ldcs(tm + i) : 0.f;
        v[j] = live ? __ldcs(tv + i) : 0.f;
    }
    AdamScalars s = a.s;
    if (t.n & kNoDecay) s.decay = 1.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) adamw_elem(__fmul_rn(g[j], factor), p[j], m[j], v[j], s);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t i = begin + 32 * j;
        if (i >= n) break;
        t.master[i] = p[j];
        if (t.param) t.param[i] = f32_to_bf16(p[j]);
        tm[i] = m[j];
        tv[i] = v[j];
    }
}

// A ring of tiles in shared memory: one warp brings whole tiles there by bulk copies (their scales, at any 4-byte address, by
// 4-byte copies that count on the same barrier), eight warps work on a block each and write it from registers.  Arrays at
// other addresses come as the 16-byte chunks that cover the tile, each with its own offset, and go back by bulk copies too
// (step_shifted), where those chunks lie inside the tensor.  Of any other tile - a tensor's last, and its first where the
// arrays are shifted - only the place is passed on, and the warps read its blocks themselves.  402 M elements with states in
// 8 bits: 932 us (6.46 GB, 950 at the copy rate); 139 M in 32 bits 551 (558).  All arrays three elements off: 60 % and 84 %
// of the copy rate, bound by the single-element accesses to shared memory; 34 % and 58 % before, with global ones.
template <bool G32, bool Q>
struct Ring8 {
    static constexpr int kGrad = kTile * (G32 ? 4 : 2), kState = kTile * (Q ? 1 : 4);
    static constexpr int kScales = Q ? 2 * kTileBlocks * 4 : 0;
    static constexpr int kBulk = kGrad + kTile * 4 + 2 * kState;     // what an aligned tile has
    // a stage: gradients, masters, m, v, each with room for an offset, and the scales
    static constexpr int kMaster = kGrad + 16, kM = kMaster + kTile * 4 + 16, kV = kM + kState + 16, kScale = kV + kState + 16;
    static constexpr int kStage = kScale + kScales;
    static constexpr int kStages = Q ? (G32 ? 3 : 4) : 2;            // 57 to 66 KB, three CTAs per SM
};
enum { kElsewhere = 0, kInPlace = 1, kShifted = 2 };
struct Job {                         // a stage's tile
    int64_t block;                   // of the tensor
    int e;
    uint32_t how;
};
constexpr int kStepCtas = 3, kNormCtas = 4;          // resident CTAs per SM
constexpr int kWorkers = 32 * kTileBlocks, kStepThreads = kWorkers + 32;
template <bool G32, bool Q>
constexpr int kStepSmem = Ring8<G32, Q>::kStages * (Ring8<G32, Q>::kStage + (int)sizeof(Job) + 16) + 64;

__device__ __forceinline__ uint32_t offset16(const void* p) { return (uint32_t)((uintptr_t)p & 15); }

// bytes (a multiple of 16) from src to dst, both 16-byte aligned, counted on bar.
__device__ __forceinline__ void bulk(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(su32(dst)), "l"(src),
                 "r"(bytes), "r"(su32(bar))
                 : "memory");
}

// The bytes [to, to + n) from shared memory at an address that is the same modulo 16; a warp, elements of `size` bytes.  The
// caller waits until the copy has read.
__device__ __forceinline__ void write_back(uint8_t* to, const uint8_t* from, int n, int size) {
    const int lane = threadIdx.x & 31, head = (16 - (int)offset16(to)) & 15, body = (n - head) & ~15, tail = head + body;
    if (lane == 0) {
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to + head), "r"(su32(from + head)), "r"(body) : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    // what is left on either side, an element per lane
    const int at = lane * size < head ? lane * size : tail + lane * size - head;
    if (at >= n) return;
    if (size == 1) to[at] = from[at];
    else if (size == 2) *reinterpret_cast<uint16_t*>(to + at) = *reinterpret_cast<const uint16_t*>(from + at);
    else *reinterpret_cast<uint32_t*>(to + at) = *reinterpret_cast<const uint32_t*>(from + at);
}

// Waits until all eight warps have written tile number `tile` of the shifted ones.  A warp that gives up leaves the number of
// the first that it does not arrive for, so that this ends, and the same way for every warp: a tile goes back as a whole.
__device__ __forceinline__ bool all_written(uint64_t* written, const volatile uint32_t* left_at, uint32_t tile) {
    if (mbar_try_wait(written, tile & 1)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(written, tile & 1)) {
        if (*left_at <= tile || clock64() - t0 > kDrainLimit) return false;
    }
    return true;
}

// A tile whose arrays have offsets.  The eight warps read their blocks of the stage, write the results to the same places
// (the parameters to the gradients', once all have read), and four of them bring an array each back, two with its scales:
// a tile whose waits run out is left as it was.  `read` and `written`: barriers of the eight warps; `tile`: how many such
// tiles the CTA had before.  False: a wait ran out.  (With one warp for all arrays, another for every tile, 201 M elements
// three off in 8 bits take 1110 us in the place of 892.)
template <bool G32, bool Q, int CAP>
__device__ __noinline__ bool step_shifted(const Table<CAP>& a, int e, int64_t block0, uint8_t* stage, uint64_t* read, uint64_t* written,
                                          uint32_t* left_at, uint32_t tile, float factor) {
    using R = Ring8<G32, Q>;
    const Entry& t = a.t[e];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = warp * kBlock + lane;
    const int64_t block = block0 + warp, i = block0 * kBlock;
    float* scales = reinterpret_cast<float*>(stage + R::kScale);
    constexpr int kStateSize = Q ? 1 : 4;
    uint8_t* sg = stage + offset16(t.grad);
    uint8_t* sp = stage + R::kMaster + offset16(t.master);
    uint8_t* sm = stage + R::kM + offset16(t.m);
    uint8_t* sv = stage + R::kV + offset16(t.v);
    uint8_t* sb = stage + offset16(t.param);                 // where the parameters go
    float g[8], p[8], m[8], v[8];
    Codes8 c;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int k = mine + 32 * j;
        g[j] = G32 ? reinterpret_cast<const float*>(sg)[k] : bf16_to_f32(reinterpret_cast<const uint16_t*>(sg)[k]);
        p[j] = reinterpret_cast<const float*>(sp)[k];
        if (!Q) {
            m[j] = reinterpret_cast<const float*>(sm)[k];
            v[j] = reinterpret_cast<const float*>(sv)[k];
        }
    }
    if (Q) {
        auto four = [&](const uint8_t* q) { return q[mine] | (q[mine + 32] << 8) | (q[mine + 64] << 16) | ((uint32_t)q[mine + 96] << 24); };
        c = Codes8{make_uint2(four(sm), four(sm + 128)), make_uint2(four(sv), four(sv + 128)), scales[warp], scales[kTileBlocks + warp]};
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(read);
    if constexpr (Q) {
        float2 gp[4], pp[4];
        to_pairs(g, gp);
        to_pairs(p, pp);
        if (step8<5>(gp, pp, c, hash_of(a, e, block * kBlock + lane), factor, scalars8(a, t))) {
            of_pairs(pp, p);
        } else {                                 // in place, and from there into the stage like the other blocks
            step_any<G32>(a, e, block, factor);
            __syncwarp();
            Strided<G32>(t, block).load(g, p, c, block);
        }
    } else {
        AdamScalars s = a.s;
        if (t.n & kNoDecay) s.decay = 1.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) adamw_elem(__fmul_rn(g[j], factor), p[j], m[j], v[j], s);
    }
    if (!__all_sync(~0u, mbar_wait_or_look(read, tile & 1, a.wait_limit))) {
        if (lane == 0) atomicMin(left_at, tile);
        return false;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int k = mine + 32 * j;
        reinterpret_cast<float*>(sp)[k] = p[j];
        if (t.param) reinterpret_cast<uint16_t*>(sb)[k] = f32_to_bf16(p[j]);
        if (Q) {
            sm[k] = (uint8_t)((j < 4 ? c.m.x : c.m.y) >> (8 * (j & 3)));
            sv[k] = (uint8_t)((j < 4 ? c.v.x : c.v.y) >> (8 * (j & 3)));
        } else {
            reinterpret_cast<float*>(sm)[k] = m[j];
            reinterpret_cast<float*>(sv)[k] = v[j];
        }
    }
    if (Q && lane == 0) {
        scales[warp] = c.ms;
        scales[kTileBlocks + warp] = c.vs;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(written);
    if (warp >= 4) return true;
    if (!__all_sync(~0u, all_written(written, left_at, tile))) return false;
    if (warp == 0) write_back(reinterpret_cast<uint8_t*>(t.master + i), sp, kTile * 4, 4);
    if (warp == 1) write_back(static_cast<uint8_t*>(t.m) + i * kStateSize, sm, kTile * kStateSize, kStateSize);
    if (warp == 2) write_back(static_cast<uint8_t*>(t.v) + i * kStateSize, sv, kTile * kStateSize, kStateSize);
    if (warp == 3 && t.param) write_back(reinterpret_cast<uint8_t*>(t.param + i), sb, kTile * 2, 2);
    if (Q && lane < kTileBlocks) {
        if (warp == 1) t.m_scale[block0 + lane] = scales[lane];
        if (warp == 2) t.v_scale[block0 + lane] = scales[kTileBlocks + lane];
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
    return true;
}

// SHIFTS: some tensor of the list has arrays with offsets.  (With that path in it, though it is never taken, the kernel for
// others keeps fewer values in registers: 402 M elements in 8 bits, the norm before it, 1131 us for 1074.)
template <bool G32, bool Q, bool SHIFTS, int CAP>
__global__ void __launch_bounds__(kStepThreads, kStepCtas) k_adamw_tensors(const __grid_constant__ Table<CAP> a) {
    using R = Ring8<G32, Q>;
    extern __shared__ __align__(128) uint8_t ring_sh[];
    Job* jobs = reinterpret_cast<Job*>(ring_sh + R::kStages * R::kStage);
    uint64_t* full = reinterpret_cast<uint64_t*>(jobs + R::kStages);
    uint64_t* empty = full + R::kStages;
    uint64_t* read = empty + R::kStages;         // step_shifted's
    uint64_t* written = read + 1;
    uint32_t* sent = reinterpret_cast<uint32_t*>(written + 1);
    uint32_t* left_at = sent + 1;                // step_shifted's
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < R::kStages; ++i) {
            mbar_init(full + i, 33);             // the bulk copies' bytes, and what each of 32 lanes copies besides
            mbar_init(empty + i, kTileBlocks);
        }
        mbar_init(read, kTileBlocks);
        mbar_init(written, kTileBlocks);
        *left_at = ~0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    dependent_launch_prologue();
    __syncthreads();
    const float factor = a.factor ? *a.factor : 1.f;
    if (isnan(factor)) return;                   // gradients that are not finite: no step
    const uint32_t begin = blockIdx.x * a.run, end = min(a.tiles, begin + a.run);
    int at = 0;
    uint32_t round = 0;
    auto next = [&] {
        if (++at == R::kStages) {
            at = 0;
            ++round;
        }
    };
    if (warp == kTileBlocks) {
        int e = 0;
        bool ok = true;
        for (uint32_t u = begin; u < end; ++u) {
            e = find(a, u, e);
            const Entry& t = a.t[e];
            const int64_t block = (int64_t)(u - a.first[e]) * kTileBlocks, i = block * kBlock;
            const int64_t left = (t.n & kCount) - i;
            const uint32_t how = t.n & kAligned ? (left >= kTile ? kInPlace : kElsewhere)
                                 : SHIFTS && block > 0 && left >= kTile + 16   ? kShifted
                                                                               : kElsewhere;
            if (round > 0 && !(ok = __all_sync(~0u, mbar_wait_or_look(empty + at, (round & 1) ^ 1, a.wait_limit)))) break;
            uint8_t* to = ring_sh + at * R::kStage;
            if (lane == 0) jobs[at] = Job{block, e, how};
            if (how != kElsewhere) {
                if (lane == 0) {
                    const uint8_t *g = static_cast<const uint8_t*>(t.grad) + i * (G32 ? 4 : 2), *p = reinterpret_cast<const uint8_t*>(t.master + i),
                                  *m = static_cast<const uint8_t*>(t.m) + i * (Q ? 1 : 4), *v = static_cast<const uint8_t*>(t.v) + i * (Q ? 1 : 4);
                    if (!SHIFTS || how == kInPlace) {
                        mbar_expect_tx(full + at, R::kBulk);
                        bulk(to, g, R::kGrad, full + at);
                        bulk(to + R::kMaster, p, kTile * 4, full + at);
                        bulk(to + R::kM, m, R::kState, full + at);
                        bulk(to + R::kV, v, R::kState, full + at);
                    } else {                     // the chunks that cover them: one more where there is an offset
                        auto more = [](const void* q) { return offset16(q) ? 16u : 0u; };
                        mbar_expect_tx(full + at, R::kBulk + more(g) + more(p) + more(m) + more(v));
                        bulk(to, g - offset16(g), R::kGrad + more(g), full + at);
                        bulk(to + R::kMaster, p - offset16(p), kTile * 4 + more(p), full + at);
                        bulk(to + R::kM, m - offset16(m), R::kState + more(m), full + at);
                        bulk(to + R::kV, v - offset16(v), R::kState + more(v), full + at);
                    }
                }
                if (Q && lane < 2 * kTileBlocks) {
                    const float* from = (lane < kTileBlocks ? t.m_scale : t.v_scale) + block + lane % kTileBlocks;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(su32(to + R::kScale + lane * 4)), "l"(from) : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(su32(full + at)) : "memory");
            } else {
                if (lane == 0) mbar_arrive(full + at);
                mbar_arrive(full + at);
            }
            __syncwarp();
            next();
        }
        if (lane == 0) *sent = round * R::kStages + at;
        if (!ok && lane == 0) atomicCAS(a.error, 0u, ZS_DEVERR_TENSORS_WAIT);
    } else {
        uint32_t shifted = 0;                    // tiles so far
        for (uint32_t u = begin; u < end; ++u, next()) {
            if (!__all_sync(~0u, mbar_wait_or_look(full + at, round & 1, a.wait_limit))) {
                if (lane == 0) {
                    atomicCAS(a.error, 0u, ZS_DEVERR_TENSORS_WAIT);
                    if (SHIFTS) atomicMin(left_at, shifted);
                }
                break;
            }
            const Job job = jobs[at];
            const Entry& t = a.t[job.e];
            const int64_t block = job.block + warp, i = block * kBlock + lane * 8;
            if (SHIFTS && job.how == kShifted) {
                if (!step_shifted<G32, Q>(a, job.e, job.block, ring_sh + at * R::kStage, read, written, left_at, shifted, factor)) {
                    if (lane == 0) atomicCAS(a.error, 0u, ZS_DEVERR_TENSORS_WAIT);
                    break;
                }
                if (lane == 0) mbar_arrive(empty + at);
                ++shifted;
                continue;
            }
            if (job.how == kElsewhere) {
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + at);
                if (block * kBlock < (t.n & kCount)) {
                    if constexpr (Q) step_strided<G32>(a, job.e, block, factor);
                    else step_strided32<G32>(a, job.e, block, factor);
                }
                continue;
            }
            const uint8_t* stage = ring_sh + at * R::kStage;
            const int mine = warp * kBlock + lane * 8;
            float g[8], p[8];
            auto floats = [](const uint8_t* q, float (&f)[8]) {
                const float4 x = reinterpret_cast<const float4*>(q)[0], y = reinterpret_cast<const float4*>(q)[1];
                f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
                f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
            };
            if constexpr (G32) floats(stage + mine * 4, g);
            else unpack(BfVec<8>{*reinterpret_cast<const uint4*>(stage + mine * 2)}, g);
            floats(stage + R::kMaster + mine * 4, p);
            if constexpr (Q) {
                const float* scales = reinterpret_cast<const float*>(stage + R::kScale);
                Codes8 c{*reinterpret_cast<const uint2*>(stage + R::kM + mine), *reinterpret_cast<const uint2*>(stage + R::kV + mine), scales[warp],
                         scales[kTileBlocks + warp]};
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + at);
                float2 gp[4], pp[4];
                to_pairs(g, gp);
                to_pairs(p, pp);
                if (!step8<0>(gp, pp, c, hash_of(a, job.e, i), factor, scalars8(a, t))) {
                    step_any<G32>(a, job.e, block, factor);
                    continue;
                }
                of_pairs(pp, p);
                __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i), c.m);
                __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i), c.v);
                if (lane == 0) {
                    t.m_scale[block] = c.ms;
                    t.v_scale[block] = c.vs;
                }
            } else {
                float m[8], v[8];
                floats(stage + R::kM + mine * 4, m);
                floats(stage + R::kV + mine * 4, v);
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + at);
                AdamScalars s = a.s;
                if (t.n & kNoDecay) s.decay = 1.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) adamw_elem(__fmul_rn(g[j], factor), p[j], m[j], v[j], s);
                store8(static_cast<float*>(t.m) + i, m);
                store8(static_cast<float*>(t.v) + i, v);
            }
            store8(t.master + i, p);
            if (t.param) st_bf<8>(t.param + i, pack(p));
        }
    }
    if (SHIFTS && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncthreads();
    if (warp == 0) ring_settled(full, R::kStages, *sent);        // no copy is under way when the CTA goes
}

// ------------------------------------------------------------------ the gradients' norm

// Sum over the CTA's 256 threads, in thread 0.
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double sh[8];
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(~0u, x, k);
    if (lane == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
    x = lane < 8 ? sh[lane] : 0.0;
#pragma unroll
    for (int k = 4; k > 0; k >>= 1) x += __shfl_xor_sync(~0u, x, k);
    return x;
}

// A CTA's sum among the partial ones: the fp64 number in two words, as sums of fp32 squares go past fp32's range.
__device__ __forceinline__ double partial_sum(const float* partials, int i) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(partials) + 2 * i;
    return __hiloint2double((int)p[1], (int)p[0]);
}
__device__ __forceinline__ void keep_partial_sum(float* partials, int i, double sum) {
    uint32_t* p = reinterpret_cast<uint32_t*>(partials) + 2 * i;
    p[0] = (uint32_t)__double2loint(sum);
    p[1] = (uint32_t)__double2hiint(sum);
}

// The norm and the factor from the sum of squares.
__device__ __forceinline__ void norm_and_factor(double sum, float max_norm, float* out) {
    // the root of the nearest fp32 number, corrected by what that leaves (a division in fp64 takes longer than the rest);
    // sums past fp32's range are scaled into it, finite ones are below 2^128 times the number of tiles and lanes
    const bool large = sum > 0x1p120;
    const double s = large ? sum * 0x1p-128 : sum;
    const float r = sqrtf((float)s);
    const bool inside = r > 0.f && isfinite(r);
    const float root = inside ? (float)((double)r + (s - (double)r * r) * (double)(0.5f / r)) : r;
    const float norm = large ? root * 0x1p64f : root;
    out[0] = norm;
    // not finite: no factor, and a step given it is not taken
    out[1] = isfinite(norm) ? fminf(__fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f)), 1.f) : __int_as_float(0x7fffffff);
}

// A lane adds a tile's 64 squares in fp32, and those sums in fp64 (one fp64 addition per block of 256 alone took the
// time of twice the bytes: 402 M bf16 gradients 210 us, now 117; 118 at the copy rate).  The CTAs' sums (as many as the caller has room for, each of
// its own blocks, so the same bits every time) are kept in two words each and added by one CTA.
template <bool G32, int CAP>
__global__ void __launch_bounds__(256, kNormCtas) k_grad_norm(const __grid_constant__ Table<CAP> a) {
    dependent_launch_prologue();
    const int lane = threadIdx.x & 31;
    const uint32_t warps = (uint32_t)(gstride() >> 5);
    double sum = 0.0;
    int e = 0;
    for (uint32_t u = (uint32_t)(gtid() >> 5); u < a.tiles; u += warps) {
        e = find(a, u, e);
        // tiles from the tensor's first element at 8 elements' bytes on; the first tile takes those before it along
        const Entry& t = a.t[e];
        constexpr int kSize = G32 ? 4 : 2;
        const int64_t n = t.n & kCount, begin = (int64_t)(u - a.first[e]) * kTile;
        const int64_t head = min(n, (int64_t)((0 - (uintptr_t)t.grad) & (8 * kSize - 1)) / kSize), left = n - head - begin;
        const uint8_t* from = static_cast<const uint8_t*>(t.grad) + (head + begin) * kSize;
        float q[kTileBlocks];
        auto squares = [](const float (&g)[8]) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(g[j], g[j], s);
            return s;
        };
        if (left >= kTile) {
#pragma unroll
            for (int b = 0; b < kTileBlocks; ++b) {
                float g[8];
                load_grad8<G32>(from, b * kBlock + lane * 8, g);
                q[b] = squares(g);
            }
        } else {
#pragma unroll
            for (int b = 0; b < kTileBlocks; ++b) {
                const int at = b * kBlock + lane * 8;
                float g[8];
                if (at + 8 <= left) {
                    load_grad8<G32>(from, at, g);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[j] = at + j < left ? load_grad<G32>(from, at + j) : 0.f;
                }
                q[b] = squares(g);
            }
        }
        if (begin == 0 && lane < head) {
            const float g = load_grad<G32>(t.grad, lane);
            q[0] = fmaf(g, g, q[0]);
        }
        sum += ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        if (a.add) sum += partial_sum(a.partials, (int)blockIdx.x);
        keep_partial_sum(a.partials, (int)blockIdx.x, sum);
        if (a.out) norm_and_factor(sum, a.max_norm, a.out);          // the only CTA
    }
}

__global__ void __launch_bounds__(256) k_grad_norm_end(const float* partials, int n, float max_norm, float* out) {
    dependent_launch_prologue();
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += 256) sum += partial_sum(partials, i);
    sum = block_sum(sum);
    if (threadIdx.x == 0) norm_and_factor(sum, max_norm, out);
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

// Whether the step's tiles are copied as they are, and values written eight at a time.
bool in_place(const zs_tensor& t, int state_bits) {
    const uintptr_t state = state_bits == 8 ? 16 : 32;
    return aligned(t.grad, 16) && aligned(t.master, 32) && aligned(t.param, 16) && aligned(t.m, state) && aligned(t.v, state);
}

// Calls launch(table, first) for the tensors, as many at a time as a launch's parameters hold.
template <int CAP, typename F>
cudaError_t by_table(const zs_tensor* tensors, int count, int state_bits, uint32_t seed, Table<CAP>& a, F launch) {
    bool first = true;
    int i = 0;
    do {
        a.count = 0;
        uint64_t tiles = 0;
        for (; i < count && a.count < CAP; ++i) {
            const zs_tensor& t = tensors[i];
            if (t.n == 0) continue;
            const uint64_t more = (uint64_t)(t.n + kTile - 1) / kTile;
            if (a.count && tiles + more > 0x7fffffffu) break;
            Entry& e = a.t[a.count];
            e = Entry{t.grad, t.master, (uint16_t*)t.param, t.m, t.v, t.m_scale, t.v_scale, t.n};
            if (in_place(t, state_bits)) e.n |= kAligned;
            if (t.no_decay) e.n |= kNoDecay;
            a.first[a.count] = (uint32_t)tiles;
            a.key[a.count] = mix(seed + 0x9e3779b9u * ((uint32_t)i + 1));
            tiles += more;
            ++a.count;
        }
        a.tiles = (uint32_t)tiles;
        if (a.count || first) {
            const cudaError_t rc = launch(a, first);
            if (rc != cudaSuccess) return rc;
        }
        first = false;
    } while (i < count);
    return cudaSuccess;
}


// Tiles of a CTA, at most.  CTAs that end and are replaced take the work as the SMs get through it, which a fixed share for
// each does not (402 M elements with states in 8 bits, the norm before it: 1121, 1074, 1087 us with 4, 8 and 16 tiles, and
// about 150 more in fixed shares.  139 M with states in 32 bits: 549, 551, 574 with 2, 3 and 8, and 65 more).
constexpr uint32_t kRun8 = 8, kRun32 = 3;

template <bool G32, bool Q, bool SHIFTS, int CAP>
cudaError_t launch_step(Table<CAP>& t, cudaStream_t st) {
    constexpr int smem = kStepSmem<G32, Q>;
    static_assert(kStepCtas * (smem + 1024) <= 228 * 1024, "resident CTAs");
    static std::atomic<uint64_t> ready{0};
    const auto kern = k_adamw_tensors<G32, Q, SHIFTS, CAP>;
    const cudaError_t e = ready_once(ready, (const void*)kern, smem);
    if (e != cudaSuccess) return e;
    const uint32_t room = (uint32_t)q8_host::sm_count() * kStepCtas, most = Q ? kRun8 : kRun32, run = t.tiles / (room * 4);
    t.run = run < 1 ? 1 : run < most ? run : most;
    return launch_kernel(kern, dim3((t.tiles + t.run - 1) / t.run), dim3(kStepThreads), smem, st, t);
}

template <bool G32, bool Q, int CAP>
cudaError_t step_tensors(const zs_tensor* tensors, int count, uint32_t seed, Table<CAP>& a, cudaStream_t st) {
    return by_table<CAP>(tensors, count, Q ? 8 : 32, seed, a, [&](Table<CAP>& t, bool) {
        if (!t.count) return cudaSuccess;
        bool shifts = false;
        for (int i = 0; i < t.count; ++i) shifts |= !(t.t[i].n & kAligned) && (t.t[i].n & kCount) > 2 * kTile;
        return shifts ? launch_step<G32, Q, true>(t, st) : launch_step<G32, Q, false>(t, st);
    });
}

template <int CAP>
cudaError_t step_list(const zs_tensor* tensors, int count, bool g32, bool q, uint32_t seed, const AdamScalars& s, const float* factor,
                     cudaStream_t st) {
    Table<CAP> a;
    a.s = s;
    a.inv_root = (float)(1.0 / (double)s.sqrt_bc2);
    a.eps = s.eps > 0.f && s.eps < FLT_MIN ? FLT_MIN : s.eps;
    a.one = 1.f;
    a.factor = factor;
    a.wait_limit = wait_limit().load(std::memory_order_relaxed);
    if (const cudaError_t e = error_word(&a.error); e != cudaSuccess) return e;
    return g32 ? (q ? step_tensors<true, true>(tensors, count, seed, a, st) : step_tensors<true, false>(tensors, count, seed, a, st))
               : (q ? step_tensors<false, true>(tensors, count, seed, a, st) : step_tensors<false, false>(tensors, count, seed, a, st));
}

template <bool G32, int CAP>
cudaError_t norm_tensors(const zs_tensor* tensors, int count, float* partials, int n_partials, float max_norm, float* out, cudaStream_t st) {
    Table<CAP> a;
    a.partials = partials;
    a.max_norm = max_norm;
    a.out = n_partials == 1 ? out : nullptr;     // overwritten by later launches, if there are any
    return by_table<CAP>(tensors, count, 32, 0, a, [&](Table<CAP>& t, bool first) {
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
    bool any = false;
    for (int i = 0; i < n_tensors; ++i) any |= tensors[i].n > 0;
    if (!any) return ZS_OK;
    const cudaStream_t st = (cudaStream_t)stream;
    return cuda_status(fn, n_tensors <= zs::kTableFew
                               ? zs::step_list<zs::kTableFew>(tensors, n_tensors, grad_bytes == 4, state_bits == 8, seed, s, factor, st)
                               : zs::step_list<zs::kTableMost>(tensors, n_tensors, grad_bytes == 4, state_bits == 8, seed, s, factor, st));
}

extern "C" int zs_grad_norm(const zs_tensor* tensors, int32_t n_tensors, int32_t grad_bytes, float max_norm, float* partials,
                            int64_t n_partials, float* out, void* stream) {
    static const char* fn = "zs_grad_norm";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    if (!(max_norm > 0.f) || !std::isfinite(max_norm)) return fail(fn, "max_norm must be positive and finite");
    if (!partials || !zs::aligned(partials, 4)) return fail(fn, "partials is NULL or not 4-byte aligned");
    if (n_partials < 2) return fail(fn, "n_partials must be at least 2");
    if (!out || !zs::aligned(out, 4)) return fail(fn, "out is NULL or not 4-byte aligned");
    ZS_Q8_TRY(zs::check_list(fn, tensors, n_tensors, grad_bytes, 32, false));
    const cudaStream_t st = (cudaStream_t)stream;
    int64_t tiles = 0;
    for (int i = 0; i < n_tensors; ++i) tiles += (tensors[i].n + zs::kTile - 1) / zs::kTile;
    int64_t most = (int64_t)sm_count() * zs::kNormCtas, ctas = (tiles + 7) / 8;
    if (most > n_partials / 2) most = n_partials / 2;
    const int n = (int)(ctas < 1 ? 1 : ctas < most ? ctas : most);
    const bool few = n_tensors <= zs::kTableFew;
    cudaError_t e;
    if (grad_bytes == 4) e = few ? zs::norm_tensors<true, zs::kTableFew>(tensors, n_tensors, partials, n, max_norm, out, st) : zs::norm_tensors<true, zs::kTableMost>(tensors, n_tensors, partials, n, max_norm, out, st);
    else e = few ? zs::norm_tensors<false, zs::kTableFew>(tensors, n_tensors, partials, n, max_norm, out, st) : zs::norm_tensors<false, zs::kTableMost>(tensors, n_tensors, partials, n, max_norm, out, st);
    if (e == cudaSuccess && n > 1) e = zs::launch_kernel(zs::k_grad_norm_end, dim3(1), dim3(256), 0, st, (const float*)partials, n, max_norm, out);
    return cuda_status(fn, e);
}
