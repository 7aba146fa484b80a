// Product of two 8-bit matrices (zs_q8_matmul): out = scale * P Q^T (+ out) over their common columns.
//
// tcgen05.mma kind::mxf8f6f4 multiplies e4m3 codes and applies one e8m0 scale per row and 32 columns
// inside the tensor core; the format's scales are per 128 columns, so the four K = 32 instructions of a
// 128-column block name the same scale byte.  One 32-bit word of tensor memory holds a row's scales of
// four blocks (the instruction descriptor's scale id picks the byte), so scales are fetched once per
// 512 columns.
//
// Roles of a CTA's warps: 0 loads tiles of codes (TMA, 128-byte swizzle) into a ring of stages; 1 issues
// the scale copies and the products (one thread); 2 fetches scale bytes and lays them out as the scale
// copy wants them; 3 holds the tensor memory allocation; 4-7 read the accumulator and write the result.
#include <cuda.h>

#include <atomic>
#include <mutex>

#include "q8.cuh"

namespace zs {

namespace {

constexpr int kMmThreads = 256;
constexpr int kMaxDevices = 64;

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(su32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity, long long limit) {
    if (mbar_try_wait(b, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(b, parity)) {
        if (clock64() - t0 > limit) return false;
    }
    return true;
}

// Tile of codes: columns x .. x + 127, rows y ..; x is a multiple of 128, so the copy starts on a
// 16-byte boundary as it must.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            su32(dst)),
        "l"((uint64_t)map), "r"(x), "r"(y), "r"(su32(bar))
        : "memory");
}

// Shared-memory operand: rows of 128 bytes, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Shared-memory source of a scale copy: 32 rows of 16 bytes, no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t scales_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

__device__ __forceinline__ void tmem_copy_scales(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// ------------------------------------------------------------------ the CTA pair (cta_group::2)

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of the cluster; orders shared-memory writes before it against reads after it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Cluster address of this CTA's shared-memory address in CTA `rank`.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(su32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(su32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
// mbar_wait for a barrier at which threads of the other CTA arrive (what copies and products signal needs
// no wider scope than the CTA's: their data never passes through this thread's loads).
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* b, uint32_t parity, long long limit) {
    if (mbar_try_wait_cluster(b, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait_cluster(b, parity)) {
        if (clock64() - t0 > limit) return false;
    }
    return true;
}
// tma_load whose bytes count on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(su32(dst)),
        "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Into both CTAs' tensor memory, each from its own shared memory.
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_scaled_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                                uint32_t sfb, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
        : "memory");
}
// Arrives at the barrier of this offset in both CTAs.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(su32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// 32 columns of this warp's 32 accumulator rows.
__device__ __forceinline__ void tmem_load32(uint32_t tmem, float (&f)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(tmem));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
}

// Position in a ring of stages: the stage and how often the ring has gone round.
struct Ring {
    int at = 0;
    uint32_t round = 0;
    __device__ __forceinline__ uint32_t parity() const { return round & 1; }
    __device__ __forceinline__ void next(int stages) {
        if (++at == stages) {
            at = 0;
            ++round;
        }
    }
};

struct MmArgs {
    const uint8_t *sp, *sq;      // scales of the P and Q operands
    int64_t ldsp, ldsq;
    int rows_p, rows_q;          // valid rows
    int kblocks, blocks;         // 128-column blocks of the sum (the products stop at the last; scales exist for it)
    int tiles_q;                 // tiles of Q: tile t is P tile t / tiles_q, Q tile t % tiles_q
    uint16_t* out;
    int64_t ldo;
    int transposed;              // 0: out[p][q], 1: out[q][p]
    int wide;                    // rows of out take 16-byte stores
    float scale;
    int first;
    unsigned int* error;
    long long wait_limit;
};

template <int BN, int STAGES>
struct MmShape {
    static constexpr int kStageBytes = 128 * 128 + BN * 128;
    static constexpr int kQChunks = (BN + 127) / 128;
    static constexpr int kScaleBytes = 512 * (1 + kQChunks);
    static constexpr int kScaleCols = 4 * (1 + kQChunks);
    static constexpr int kTmemCols = BN + 2 * kScaleCols <= 32 ? 32 : BN + 2 * kScaleCols <= 64 ? 64
                                     : BN + 2 * kScaleCols <= 128 ? 128 : BN + 2 * kScaleCols <= 256 ? 256 : 512;
    static constexpr int kSmem = 1024 + STAGES * kStageBytes + 2 * kScaleBytes + 256;
};

// One row's scale bytes, kBatch groups of four blocks at a time.  Rows of scales start at any byte, so a
// group is cut out of two neighbouring aligned words; every word is loaded once.  Words that reach over
// either end of the matrix of scales are put together from its bytes.  Blocks past the row's last give
// scale byte 0, and so do rows past the matrix (their codes read as 0).
constexpr int kBatch = 4;
struct ScaleRow {
    const uint8_t *at, *lo, *hi;     // word to load next; the matrix of scales
    uint32_t w[kBatch + 1], shift;
    int left;                        // blocks from the current batch on
    __device__ __forceinline__ uint32_t load() {
        const uint8_t* p = at;
        at += 4;
        if (p >= lo && p + 4 <= hi) return *reinterpret_cast<const uint32_t*>(p);
        uint32_t x = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (p + k >= lo && p + k < hi) x |= (uint32_t)p[k] << (8 * k);
        return x;
    }
    __device__ __forceinline__ void fill() {                 // w[1 ..], after w[0]
#pragma unroll
        for (int j = 1; j <= kBatch; ++j) w[j] = left > 4 * (j - 1) ? load() : 0;
    }
    // Row `row` of s from block `first` on, `blocks` of them; the rows have `all`.
    __device__ __forceinline__ void start(const uint8_t* s, int64_t ld, int64_t row, int rows, int first, int blocks, int all) {
        left = row < rows ? blocks : 0;
        lo = s;
        hi = left ? s + (int64_t)(rows - 1) * ld + all : s;
        const uint8_t* p = left ? s + row * ld + first : s;
        shift = (uint32_t)((uintptr_t)p & 3) * 8;
        at = (const uint8_t*)((uintptr_t)p & ~(uintptr_t)3);
        w[0] = load();
        fill();
    }
    __device__ __forceinline__ uint32_t take(int j) const {
        const uint32_t x = __funnelshift_r(w[j], w[j + 1], shift);
        const int n = left - 4 * j;
        return n >= 4 ? x : n > 0 ? x & ((1u << (8 * n)) - 1) : 0;
    }
    __device__ __forceinline__ void advance() {
        left -= 4 * kBatch;
        w[0] = w[kBatch];
        fill();
    }
};

__device__ __forceinline__ uint32_t scale_word(const uint8_t* s, int64_t ld, int64_t row, int rows, int group, int blocks) {
    if (row >= rows) return 0;
    const uint8_t* p = s + row * ld + group * 4;
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (group * 4 + k < blocks) w |= (uint32_t)p[k] << (8 * k);
    return w;
}

template <int BN, int STAGES>
__global__ void __launch_bounds__(kMmThreads, 1) k_q8_matmul(const __grid_constant__ CUtensorMap map_p,
                                                             const __grid_constant__ CUtensorMap map_q,
                                                             const __grid_constant__ MmArgs a) {
    using S = MmShape<BN, STAGES>;
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (su32(raw) & 1023)) & 1023);
    uint8_t* scale_sh = base + STAGES * S::kStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(scale_sh + 2 * S::kScaleBytes);
    uint64_t* empty = full + STAGES;
    uint64_t* sfull = empty + STAGES;
    uint64_t* sempty = sfull + 2;
    uint64_t* done = sempty + 2;                 // the accumulator is complete
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(done + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull + i, 1);
            mbar_init(sempty + i, 1);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    dependent_launch_prologue();
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_at)),
                     "r"((uint32_t)S::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    const uint32_t tmem_scales = tmem + BN;
    const int tp = blockIdx.x / a.tiles_q, tq = blockIdx.x - tp * a.tiles_q;
    const int p0 = tp * 128, q0 = tq * BN;
    const int groups = (a.kblocks + 3) / 4;

    if (warp == 0 && lane == 0) {
        int issued = 0;
        for (; issued < a.kblocks; ++issued) {
            const int s = issued % STAGES;
            if (issued >= STAGES && !mbar_wait(empty + s, ((issued / STAGES) - 1) & 1, a.wait_limit)) {
                atomicCAS(a.error, 0u, ZS_DEVERR_MATMUL_WAIT);
                for (int k = issued - STAGES; k < issued; ++k)       // let the copies in flight land
                    mbar_wait(full + k % STAGES, (k / STAGES) & 1, a.wait_limit);
                break;
            }
            uint8_t* at = base + s * S::kStageBytes;
            mbar_expect_tx(full + s, S::kStageBytes);
            tma_load(at, &map_p, issued * 128, p0, full + s);
            tma_load(at + 128 * 128, &map_q, issued * 128, q0, full + s);
        }
    } else if (warp == 1 && lane == 0) {
        const uint32_t idesc = ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24);
        bool ok = true;
        for (int kb = 0; kb < a.kblocks && ok; ++kb) {
            const int s = kb % STAGES, g = kb >> 2, slot = g & 1;
            const uint32_t sfa = tmem_scales + slot * S::kScaleCols, sfb = sfa + 4;
            if ((kb & 3) == 0) {
                if (!(ok = mbar_wait(sfull + slot, (g >> 1) & 1, a.wait_limit))) break;
                tc_fence_after();
                const uint32_t at = su32(scale_sh + slot * S::kScaleBytes);
                tmem_copy_scales(sfa, scales_desc(at));
#pragma unroll
                for (int c = 0; c < S::kQChunks; ++c) tmem_copy_scales(sfb + 4 * c, scales_desc(at + 512 * (1 + c)));
                mma_commit(sempty + slot);
            }
            if (!(ok = mbar_wait(full + s, (kb / STAGES) & 1, a.wait_limit))) break;
            tc_fence_after();
            const uint32_t at = su32(base + s * S::kStageBytes);
            const uint64_t da = operand_desc(at), db = operand_desc(at + 128 * 128);
            const uint32_t id = idesc | ((uint32_t)(kb & 3) << 29) | ((uint32_t)(kb & 3) << 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_scaled(tmem, da + 2 * k, db + 2 * k, id, sfa, sfb, kb > 0 || k > 0);
            mma_commit(empty + s);
        }
        if (!ok) atomicCAS(a.error, 0u, ZS_DEVERR_MATMUL_WAIT);
        mma_commit(done);
    } else if (warp == 2) {
        for (int g = 0; g < groups; ++g) {
            const int slot = g & 1;
            uint32_t w[1 + S::kQChunks][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[0][i] = scale_word(a.sp, a.ldsp, (int64_t)p0 + lane + 32 * i, a.rows_p, g, a.blocks);
#pragma unroll
            for (int c = 0; c < S::kQChunks; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = c * 128 + lane + 32 * i;
                    w[1 + c][i] = r < BN ? scale_word(a.sq, a.ldsq, (int64_t)q0 + r, a.rows_q, g, a.blocks) : 0;
                }
            bool ok = true;
            if (g >= 2) ok = mbar_wait(sempty + slot, ((g >> 1) - 1) & 1, a.wait_limit);
            if (!__all_sync(~0u, ok)) {
                if (lane == 0) atomicCAS(a.error, 0u, ZS_DEVERR_MATMUL_WAIT);
                break;
            }
            uint4* at = reinterpret_cast<uint4*>(scale_sh + slot * S::kScaleBytes);
#pragma unroll
            for (int c = 0; c < 1 + S::kQChunks; ++c) at[c * 32 + lane] = make_uint4(w[c][0], w[c][1], w[c][2], w[c][3]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull + slot);
        }
    } else if (warp >= 4) {
        const bool ok = mbar_wait(done, 0, a.wait_limit + a.wait_limit);
        if (!__all_sync(~0u, ok)) {
            if (lane == 0) atomicCAS(a.error, 0u, ZS_DEVERR_MATMUL_WAIT);
        } else {
            tc_fence_after();
            const int sub = warp - 4;
            const int64_t p = (int64_t)p0 + sub * 32 + lane;
#pragma unroll 1
            for (int c = 0; c < BN; c += 32) {
                float f[32];
                if (q0 + c >= a.rows_q) break;
                tmem_load32(tmem + ((uint32_t)(sub * 32) << 16) + c, f);
                const int n = a.rows_q - q0 - c < (BN < 32 ? BN : 32) ? a.rows_q - q0 - c : (BN < 32 ? BN : 32);
                if (p >= a.rows_p) continue;
                if (a.transposed) {
                    uint16_t* o = a.out + (int64_t)(q0 + c) * a.ldo + p;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < n) {
                            const float old = a.first ? 0.f : bf16_to_f32(o[j * a.ldo]);
                            o[j * a.ldo] = f32_to_bf16(fmaf(f[j], a.scale, old));
                        }
                } else {
                    uint16_t* o = a.out + p * a.ldo + q0 + c;
                    if (a.wide && n == 32) {
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            float e[8], old[8];
                            if (!a.first) unpack(BfVec<8>{reinterpret_cast<const uint4*>(o)[v]}, old);
#pragma unroll
                            for (int i = 0; i < 8; ++i) e[i] = fmaf(f[v * 8 + i], a.scale, a.first ? 0.f : old[i]);
                            reinterpret_cast<uint4*>(o)[v] = pack(e).w;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j < n) {
                                const float old = a.first ? 0.f : bf16_to_f32(o[j]);
                                o[j] = f32_to_bf16(fmaf(f[j], a.scale, old));
                            }
                    }
                }
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)S::kTmemCols));
    }
}

// ------------------------------------------------------------------ large products: a persistent CTA pair per tile

// Tile of 256 P rows x 256 Q rows per pair of CTAs.  Each CTA loads its 128 P rows and half of the Q rows
// (32 KB per 128 columns; the tensor cores read the other half of Q from the other CTA), one thread of the
// leading CTA issues the products for both, and each CTA keeps 128 x 256 fp32 accumulators in its own
// tensor memory.  The pairs are persistent.  The accumulator takes half the tensor memory and the scales
// some of the rest, so it is not doubled: the eight warps that read it move it into registers as bf16,
// release it, and store while the next tile's products run.
constexpr int kPairThreads = 448;
constexpr int kPairN = 256;
constexpr int kPairStages = 6;
constexpr int kPairStageBytes = 128 * 128 + (kPairN / 2) * 128;
constexpr int kPairScaleBytes = 512 * 3;
constexpr int kPairSlots = 2;         // batches of scales in flight
constexpr int kPairSmem = 1024 + kPairStages * kPairStageBytes + kPairSlots * kBatch * kPairScaleBytes + 256;
constexpr int kPairGroup = 8;        // P tiles that share the same Q tiles at about the same time

__device__ __forceinline__ void store_pairs16(uint16_t* o, const uint32_t* w) {      // 16 bf16 values, 32-byte aligned
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_q8_matmul_pair(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                     const __grid_constant__ MmArgs a) {
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (su32(raw) & 1023)) & 1023);
    uint8_t* scale_sh = base + kPairStages * kPairStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(scale_sh + kPairSlots * kBatch * kPairScaleBytes);   // leader: both CTAs' tiles landed
    uint64_t* empty = full + kPairStages;        // each CTA: the products have read the stage
    uint64_t* sfull = empty + kPairStages;       // leader: both CTAs' scales are in shared memory
    uint64_t* sempty = sfull + kPairSlots;       // each CTA: they are copied out
    uint64_t* done = sempty + kPairSlots;        // each CTA: the accumulator is complete
    uint64_t* acc_free = done + 1;               // leader: both CTAs' accumulators are read
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(acc_free + 1);
    uint32_t* gave_up = tmem_at + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < kPairSlots; ++i) {
            mbar_init(sfull + i, 8);             // the four scale warps of both CTAs
            mbar_init(sempty + i, 1);
        }
        mbar_init(done, 1);
        mbar_init(acc_free, 16);                 // the eight reading warps of both CTAs
        *gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    dependent_launch_prologue();
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_at)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_at, tmem_scales = tmem + kPairN;
    const int groups = (a.kblocks + 3) / 4;
    const int tiles_p = (a.rows_p + 255) / 256;
    const int64_t tiles = (int64_t)tiles_p * a.tiles_q;
    const int64_t first_tile = blockIdx.x >> 1, step = gridDim.x >> 1;
    // tile t: kPairGroup P tiles at a time, within them Q tile by Q tile
    auto place = [&](int64_t t, int& p0, int& q0) {
        const int64_t per = (int64_t)kPairGroup * a.tiles_q;
        const int g = (int)(t / per), in = (int)(t - g * per);
        const int width = tiles_p - g * kPairGroup < kPairGroup ? tiles_p - g * kPairGroup : kPairGroup;
        p0 = (g * kPairGroup + in % width) * 256;
        q0 = (in / width) * kPairN;
    };
    auto fail = [&] {
        atomicExch(gave_up, 1u);
        atomicCAS(a.error, 0u, ZS_DEVERR_MATMUL_WAIT);
    };

    if (warp == 0 && lane == 0) {
        Ring ring;
        bool ok = true;
        for (int64_t t = first_tile; t < tiles && ok; t += step) {
            int p0, q0;
            place(t, p0, q0);
            for (int kb = 0; kb < a.kblocks; ++kb) {
                if (ring.round > 0 && !(ok = mbar_wait(empty + ring.at, ring.parity() ^ 1, a.wait_limit))) break;
                uint8_t* at = base + ring.at * kPairStageBytes;
                const uint32_t bar = at_rank(full + ring.at, 0);
                if (rank == 0) mbar_expect_tx(full + ring.at, 2 * kPairStageBytes);
                tma_load_pair(at, &map_p, kb * 128, p0 + (int)rank * 128, bar);
                tma_load_pair(at + 128 * 128, &map_q, kb * 128, q0 + (int)rank * (kPairN / 2), bar);
                ring.next(kPairStages);
            }
        }
        if (!ok) fail();
        if (rank == 0) {                         // let every copy land before the CTAs may exit
            const bool wrapped = ring.round > 0;
            for (int k = 0; k < kPairStages; ++k) {
                if (k < ring.at) mbar_wait(full + k, ring.parity(), a.wait_limit);
                else if (wrapped) mbar_wait(full + k, ring.parity() ^ 1, a.wait_limit);
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        const uint32_t idesc = ((uint32_t)(kPairN >> 3) << 17) | (1u << 23) | ((256u >> 4) << 24);
        const uint32_t base32 = su32(base), scale32 = su32(scale_sh);
        bool ok = true;
        Ring ring, slots;
        uint32_t tile_parity = 0;
        for (int64_t t = first_tile; t < tiles && ok; t += step) {
            if (t != first_tile) {
                if (!(ok = mbar_wait_cluster(acc_free, tile_parity, a.wait_limit))) break;
                tile_parity ^= 1;
            }
            tc_fence_after();
            uint32_t sfa = 0;
            for (int kb = 0; kb < a.kblocks; ++kb) {
                if ((kb & 3) == 0) {
                    const int in = (kb >> 2) & (kBatch - 1);
                    if (in == 0) {
                        if (!(ok = mbar_wait_cluster(sfull + slots.at, slots.parity(), a.wait_limit))) break;
                        tc_fence_after();
                    }
                    const uint32_t at = scale32 + (slots.at * kBatch + in) * kPairScaleBytes;
                    sfa = tmem_scales + in * 12;
                    tmem_copy_scales_pair(sfa, scales_desc(at));
                    tmem_copy_scales_pair(sfa + 4, scales_desc(at + 512));
                    tmem_copy_scales_pair(sfa + 8, scales_desc(at + 1024));
                    if (in == kBatch - 1 || kb + 4 >= a.kblocks) {
                        mma_commit_pair(sempty + slots.at);
                        slots.next(kPairSlots);
                    }
                }
                if (!(ok = mbar_wait(full + ring.at, ring.parity(), a.wait_limit))) break;
                tc_fence_after();
                const uint32_t at = base32 + ring.at * kPairStageBytes;
                const uint64_t da = operand_desc(at), db = operand_desc(at + 128 * 128);
                const uint32_t id = idesc | ((uint32_t)(kb & 3) << 29) | ((uint32_t)(kb & 3) << 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_scaled_pair(tmem, da + 2 * k, db + 2 * k, id, sfa, sfa + 4, kb > 0 || k > 0);
                mma_commit_pair(empty + ring.at);
                ring.next(kPairStages);
            }
            if (!ok) break;
            mma_commit_pair(done);
        }
        if (!ok) fail();
    } else if (warp >= 2 && warp < 6) {
        // thread r of 128: P row r, Q rows r and 128 + r of the tile; the scale copy wants row r's word at
        // (r % 32) * 16 + (r / 32) * 4
        Ring slots;
        bool ok = true;
        const int r = threadIdx.x - 64;
        uint8_t* mine = scale_sh + (r & 31) * 16 + (r >> 5) * 4;
        for (int64_t t = first_tile; t < tiles && ok; t += step) {
            int p0, q0;
            place(t, p0, q0);
            ScaleRow row[3];
            row[0].start(a.sp, a.ldsp, (int64_t)p0 + rank * 128 + r, a.rows_p, 0, a.blocks, a.blocks);
            row[1].start(a.sq, a.ldsq, (int64_t)q0 + r, a.rows_q, 0, a.blocks, a.blocks);
            row[2].start(a.sq, a.ldsq, (int64_t)q0 + 128 + r, a.rows_q, 0, a.blocks, a.blocks);
            for (int g = 0; g < groups; g += kBatch) {
                if (slots.round > 0) ok = mbar_wait(sempty + slots.at, slots.parity() ^ 1, a.wait_limit);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
#pragma unroll
                    for (int c = 0; c < 3; ++c)
                        *reinterpret_cast<uint32_t*>(mine + (slots.at * kBatch + j) * kPairScaleBytes + c * 512) = row[c].take(j);
                // This fence waits for every load of its thread as well: the next batch's are issued after it,
                // and a batch, not a group, is handed over at a time so that their latency is paid once per
                // 2,048 columns.  (One group at a time: 383 us for 8192^3 against 297 with no scales at all.)
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(at_rank(sfull + slots.at, 0));
                slots.next(kPairSlots);
#pragma unroll
                for (int c = 0; c < 3; ++c) row[c].advance();
            }
        }
        if (!ok && lane == 0) fail();
    } else if (warp >= 6) {
        const int sub = warp & 3, half = (warp - 6) >> 2;
        const uint32_t free_bar = at_rank(acc_free, 0);
        int64_t i = 0;
        for (int64_t t = first_tile; t < tiles; t += step, ++i) {
            int p0, q0;
            place(t, p0, q0);
            bool ok = mbar_wait(done, i & 1, a.wait_limit);
            // the products of a tile may be many: wait on while the tile still makes progress is not
            // needed, a tile of 2^31 columns ends well within the limit
            if (!__all_sync(~0u, ok)) {
                if (lane == 0) fail();
                break;
            }
            tc_fence_after();
            const int64_t p = (int64_t)p0 + rank * 128 + sub * 32 + lane;
            const int qh = q0 + half * 128;
            const bool row_ok = p < a.rows_p;
            uint16_t* o = a.out + p * a.ldo + qh;
            uint32_t w[64];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float f[32];
                tmem_load32(tmem + ((uint32_t)(sub * 32) << 16) + half * 128 + c * 32, f);
                if (a.first) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[c * 16 + j] = pack_bf16x2(f[2 * j] * a.scale, f[2 * j + 1] * a.scale);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int q = qh + c * 32 + 2 * j;
                        const float lo = row_ok && q < a.rows_q ? bf16_to_f32(o[c * 32 + 2 * j]) : 0.f;
                        const float hi = row_ok && q + 1 < a.rows_q ? bf16_to_f32(o[c * 32 + 2 * j + 1]) : 0.f;
                        w[c * 16 + j] = pack_bf16x2(fmaf(f[2 * j], a.scale, lo), fmaf(f[2 * j + 1], a.scale, hi));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(free_bar);
            if (!row_ok) continue;
            const int n = a.rows_q - qh;         // valid columns of this half
            if (a.wide && n >= 128) {
#pragma unroll
                for (int v = 0; v < 8; ++v) store_pairs16(o + v * 16, w + v * 8);
            } else {
#pragma unroll
                for (int j = 0; j < 64; ++j) {
                    if (2 * j < n) o[2 * j] = (uint16_t)w[j];
                    if (2 * j + 1 < n) o[2 * j + 1] = (uint16_t)(w[j] >> 16);
                }
            }
        }
    }
    __syncthreads();
    cluster_sync();
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    }
}

// out = (first ? 0 : out): the empty sum.
__global__ void k_q8_empty_sum(uint16_t* out, int64_t ldo, int64_t m, int64_t n) {
    dependent_launch_prologue();
    for (int64_t i = gtid(); i < m * n; i += gstride()) out[(i / n) * ldo + i % n] = 0;
}

// ------------------------------------------------------------------ host

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult got;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got) != cudaSuccess ||
            got != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

// Tiles of box_rows rows x 128 bytes of an 8-bit matrix; what lies past its rows and columns reads as 0.
bool make_map(CUtensorMap* map, const Q8& q, int64_t rows, int64_t cols, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)q.ld};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, unit[2] = {1, 1};
    return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q.codes, dims, strides, box, unit,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int STAGES>
cudaError_t launch_mm(const Q8& p, const Q8& q, int64_t k, MmArgs& a, cudaStream_t st) {
    using S = MmShape<BN, STAGES>;
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(k_q8_matmul<BN, STAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    }
    CUtensorMap mp, mq;
    if (!encode_tiled() || !make_map(&mp, p, a.rows_p, k, 128) || !make_map(&mq, q, a.rows_q, k, BN)) return cudaErrorInvalidValue;
    a.tiles_q = (a.rows_q + BN - 1) / BN;
    const int64_t tiles = (int64_t)((a.rows_p + 127) / 128) * a.tiles_q;
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_kernel(k_q8_matmul<BN, STAGES>, dim3((unsigned)tiles), dim3(kMmThreads), S::kSmem, st, mp, mq, a);
}

cudaError_t launch_mm_pair(const Q8& p, const Q8& q, int64_t k, MmArgs& a, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(k_q8_matmul_pair, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    }
    CUtensorMap mp, mq;
    if (!encode_tiled() || !make_map(&mp, p, a.rows_p, k, 128) || !make_map(&mq, q, a.rows_q, k, kPairN / 2)) return cudaErrorInvalidValue;
    a.tiles_q = (a.rows_q + kPairN - 1) / kPairN;
    const int64_t tiles = (int64_t)((a.rows_p + 255) / 256) * a.tiles_q;
    const int64_t pairs = q8_host::sm_count() / 2;
    return launch_kernel(k_q8_matmul_pair, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(kPairThreads), kPairSmem, st, mp,
                         mq, a);
}

cudaError_t error_word(unsigned int** out) {
    static std::atomic<unsigned int*> cached[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && (*out = cached[dev].load(std::memory_order_acquire))) return cudaSuccess;
    e = device_error_word(out);
    if (e == cudaSuccess && dev < kMaxDevices) cached[dev].store(*out, std::memory_order_release);
    return e;
}

}  // namespace

}  // namespace zs

using namespace zs::q8_host;

extern "C" int zs_q8_matmul(const zs_q8* a, const zs_q8* b, int64_t m, int64_t n, int64_t k, float scale, int32_t first,
                            void* out, int64_t ldo, void* stream) {
    static const char* fn = "zs_q8_matmul";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::Q8 qa, qb;
    ZS_Q8_TRY(check_dim(fn, "m", m, 0));
    ZS_Q8_TRY(check_dim(fn, "n", n, 0));
    ZS_Q8_TRY(check_dim(fn, "k", k, 0));
    ZS_Q8_TRY(check_q8(fn, "a", a, m, k, false, &qa));
    ZS_Q8_TRY(check_q8(fn, "b", b, n, k, false, &qb));
    if (!std::isfinite(scale)) return fail(fn, "scale must be finite");
    ZS_Q8_TRY(check_bf16(fn, "out", out, ldo, m, n));
    if (m == 0 || n == 0) return ZS_OK;
    const cudaStream_t st = (cudaStream_t)stream;
    if (k == 0) {
        if (!first) return ZS_OK;
        const int64_t blocks = (m * n + 255) / 256;
        return cuda_status(fn, zs::launch_kernel(zs::k_q8_empty_sum, dim3((unsigned)(blocks < 4096 ? blocks : 4096)),
                                                 dim3(256), 0, st, (uint16_t*)out, ldo, m, n));
    }
    // Few rows of a: its rows become the accumulator's columns and b's rows its 128 lanes.
    const bool swap = m <= 64;
    zs::MmArgs g{};
    const zs::Q8 &p = swap ? qb : qa, &q = swap ? qa : qb;
    g.sp = p.scales;
    g.sq = q.scales;
    g.ldsp = p.lds;
    g.ldsq = q.lds;
    g.rows_p = (int)(swap ? n : m);
    g.rows_q = (int)(swap ? m : n);
    g.kblocks = g.blocks = (int)((k + 127) / 128);
    g.out = (uint16_t*)out;
    g.ldo = ldo;
    g.transposed = swap;
    g.wide = wide(out, ldo);
    g.scale = scale;
    g.first = first != 0;
    g.wait_limit = 4000000000LL;                     // ~2 s at the 2.07 GHz maximum SM clock
    ZS_Q8_TRY(cuda_status(fn, zs::error_word(&g.error)));
    cudaError_t e;
    g.wide = wide(out, ldo);
    if (!swap && m >= 192 && n >= 192 && ((m + 255) / 256) * ((n + 255) / 256) >= 24) {
        g.wide = ((uintptr_t)out & 31) == 0 && (ldo & 15) == 0;
        e = zs::launch_mm_pair(p, q, k, g, st);
    } else if (g.rows_q <= 32) e = zs::launch_mm<32, 6>(p, q, k, g, st);
    else if (g.rows_q <= 64) e = zs::launch_mm<64, 6>(p, q, k, g, st);
    else e = zs::launch_mm<128, 6>(p, q, k, g, st);
    return cuda_status(fn, e);
}
