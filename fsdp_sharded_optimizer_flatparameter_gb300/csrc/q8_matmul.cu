// Product of two 8-bit matrices (zs_q8_matmul): out = scale * P Q^T (+ out) over their common columns.
//
// tcgen05.mma kind::mxf8f6f4 multiplies e4m3 codes and applies one e8m0 scale per row and 32 columns
// inside the tensor core; the format's scales are per 128 columns, so the four K = 32 instructions of a
// 128-column block name the same scale byte.  One 32-bit word of tensor memory holds a row's scales of
// four blocks (the instruction descriptor's scale id picks the byte), so scales are fetched once per
// 512 columns.
//
// Roles of a CTA's warps: 0 loads tiles of codes (TMA, 128-byte swizzle) into a ring of stages; 1 issues the
// scale copies and the products; 2-5 fetch scale bytes and lay them out as the scale copy wants them (2 also
// holds the tensor memory allocation); the others, four or eight, read the accumulator and write the result.
#include "q8_tma.cuh"

namespace zs {

namespace {

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
// One thread of a converged warp.  The product and copy roles run as whole warps, and only their issue is
// one thread's: what the instructions take then sits in uniform registers.  (With the role's loop run by
// lane 0 alone, issuing one block's four products took 350 cycles instead of well under the 450 they run.)
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
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
__device__ __forceinline__ void cluster_st(uint32_t at, uint32_t x) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t cluster_ld_u32(uint32_t at) {
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
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
// A whole warp waits, and agrees on the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, long long limit) {
    return __all_sync(~0u, mbar_wait(b, parity, limit));
}
__device__ __forceinline__ bool warp_wait_or_look(uint64_t* b, uint32_t parity, long long limit) {
    return __all_sync(~0u, mbar_wait_or_look(b, parity, limit));
}
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* b, uint32_t parity, long long limit) {
    return __all_sync(~0u, mbar_wait_cluster(b, parity, limit));
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
// Arrives at the barrier of this offset in the CTAs of `mask`.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar, uint16_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(su32(bar)),
        "h"(mask)
        : "memory");
}

// 16 columns of this warp's 32 accumulator rows.
__device__ __forceinline__ void tmem_load16(uint32_t tmem, float (&f)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(tmem));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r[i]);
}

// 32 columns.
__device__ __forceinline__ void tmem_load32(uint32_t tmem, float (&f)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(tmem));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
}

// Tiled stores: a warp's 32 rows x 32 columns of bf16 from 2 KB of shared memory (64-byte swizzle) to column x and row y.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"((uint64_t)map), "r"(x), "r"(y),
                 "r"(su32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Writes 16 columns of 32 rows of the result, one row per lane in f: row r of the warp at out + r * ldo.
// `rows` and `n` are what is valid of them (the same in every lane).  With `align` 32 or 16, rows start at
// multiples of that many bytes and a lane stores its own segment (a full sector at 32).  Otherwise the
// values go through 2 KB of the warp's shared memory, so that neighbouring lanes store neighbouring
// columns: one 2-byte store per lane and row cost 15 of 27 us for 160 x 339 x 4096.  What the rows hold (not
// `first`) is read at once before anything is stored (11008 x 4096 x 2048 at an odd element: 144 us, and 539 with
// each value read and stored in turn).  Reading pieces ahead, or asking lines into L2 a tile ahead, gains nothing.
__device__ __forceinline__ void store_rows16(uint16_t* out, int64_t ldo, const float (&f)[16], int rows, int n, int align,
                                             float scale, int first, float* stage) {
    const int lane = threadIdx.x & 31;
    if (rows <= 0 || n <= 0) return;
    if (align && n >= 16) {
        if (lane >= rows) return;
        uint16_t* o = out + lane * ldo;
        uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        uint4* v = reinterpret_cast<uint4*>(o);
        if (!first) {
            const uint4 x = v[0], y = v[1];
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(fmaf(f[2 * j], scale, bf16_lo(w[j])), fmaf(f[2 * j + 1], scale, bf16_hi(w[j])));
        if (align == 32) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                         "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
        } else {
            v[0] = make_uint4(w[0], w[1], w[2], w[3]);
            v[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        return;
    }
    const int c = lane & 15;
    uint16_t* o = out + (lane >> 4) * ldo + c;
    uint32_t was[8] = {0, 0, 0, 0, 0, 0, 0, 0};      // rows lane / 16 + 4 i and + 4 i + 2
    if (!first) {
        uint32_t x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 2 * i + (lane >> 4) < rows && c < n ? o[2 * i * ldo] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) was[i] = x[2 * i] | (x[2 * i + 1] << 16);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) stage[lane * 16 + (j ^ (lane & 15))] = f[j];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4);
        const float x = (i & 1) ? bf16_hi(was[i >> 1]) : bf16_lo(was[i >> 1]);
        if (r < rows && c < n) o[2 * i * ldo] = f32_to_bf16(fmaf(stage[r * 16 + (c ^ (r & 15))], scale, x));
    }
    __syncwarp();
}
constexpr int kStoreStage = 32 * 16;             // floats of shared memory per storing warp

// Position in a ring of stages: the stage and how often the ring has gone round.
struct Ring {
    int at = 0;
    uint32_t round = 0;
    __device__ __forceinline__ uint32_t count(int stages) const { return round * stages + at; }
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
    int kblocks;                 // 128-column blocks of the sum
    int tiles_q;                 // tiles of Q
    int split;                   // CTAs that share a tile's sum
    uint16_t* out;
    int64_t ldo;
    int transposed;              // 0: out[p][q], 1: out[q][p]
    int align;                   // rows of out start at multiples of 32 or 16 bytes; 0: neither
    float scale;
    int first;
    unsigned int* error;
    long long wait_limit;
    const int* starts;           // of n_groups groups and the last one's end (the experts' products)
    int n_groups;
    int group_rows;              // rows of Q (kRowGroups), P (kFewRows) or out (kSumGroups) that a group has
    int tiled;                   // out can be written by tiled copies
    int most_tiles;              // of groups that do not overlap (kRowGroups)
};

// One row's scale bytes, kBatch groups of four blocks (16 bytes) at a time.  Rows of scales start at any
// byte, so a batch is cut out of two neighbouring aligned 16-byte chunks, and every chunk is loaded once:
// the lanes of a warp read different rows, a line each, and such loads share the shared memory's bandwidth,
// which the products and the tiles' arrival need nearly all of.  (A 4-byte load per group: 333 us for
// 8192^3.)  Chunks that reach over either end of the matrix of scales are put together from its
// bytes.  Blocks past the row's last give scale byte 0, and so do rows past the matrix (their codes read
// as 0).
constexpr int kBatch = 4;
struct ScaleRow {
    const uint8_t *at, *lo, *hi;     // chunk to load next; the matrix of scales
    uint4 c0, c1;
    uint32_t off;                    // bytes of c0 before the batch
    int left;                        // blocks from the current batch on
    __device__ __forceinline__ uint4 load() {
        const uint8_t* p = at;
        at += 16;
        if (p >= lo && p + 16 <= hi) return *reinterpret_cast<const uint4*>(p);
        uint32_t x[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (p + k >= lo && p + k < hi) x[k >> 2] |= (uint32_t)p[k] << (8 * (k & 3));
        return make_uint4(x[0], x[1], x[2], x[3]);
    }
    // Row `row` of s from block `first` on, `blocks` of them; the rows have `all`.
    __device__ __forceinline__ void start(const uint8_t* s, int64_t ld, int64_t row, int rows, int first, int blocks, int all) {
        left = row < rows ? blocks : 0;
        lo = s;
        hi = left ? s + (int64_t)(rows - 1) * ld + all : s;
        const uint8_t* p = left ? s + row * ld + first : s;
        off = (uint32_t)((uintptr_t)p & 15);
        at = (const uint8_t*)((uintptr_t)p & ~(uintptr_t)15);
        c0 = load();
        c1 = (int)(16 - off) < left ? load() : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void take(uint32_t (&w)[kBatch]) const {
        uint32_t x[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        if (off & 8) {
#pragma unroll
            for (int k = 0; k < 6; ++k) x[k] = x[k + 2];
        }
        if (off & 4) {
#pragma unroll
            for (int k = 0; k < 5; ++k) x[k] = x[k + 1];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int n = left - 4 * k;
            const uint32_t v = __funnelshift_r(x[k], x[k + 1], 8 * (off & 3));
            w[k] = n >= 4 ? v : n > 0 ? v & ((1u << (8 * n)) - 1) : 0;
        }
    }
    __device__ __forceinline__ void advance() {
        left -= 4 * kBatch;
        c0 = c1;
        if ((int)(16 - off) < left) c1 = load();
    }
};

// ------------------------------------------------------------------ small products: the sum split over a cluster

// Tile of 128 P rows x BN Q rows; the blocks of the sum are split over the CTAs of a cluster, so that a
// product with few tiles (few rows, a weight of a few thousand) still loads through every SM.  Each CTA
// keeps its part in tensor memory; the parts meet in shared memory, where every CTA adds one share of the
// tile's columns over all CTAs in rank order (the same bits in every run) and writes it.  No workspace and
// no second launch.  About 100 KB per CTA, so that one CTA's start and end overlap another's loads.
constexpr int kSplitThreads = 320;
constexpr int kSplitMost = 8;        // CTAs of a cluster
template <int BN, int STAGES>
struct SplitShape {
    static constexpr int kStageBytes = 128 * 128 + BN * 128;
    static constexpr int kScaleBytes = 1024;
    static constexpr int kScaleCols = 8;
    static constexpr int kTmemCols = BN + kBatch * kScaleCols <= 64 ? 64 : BN + kBatch * kScaleCols <= 128 ? 128 : 256;
    static constexpr int kSmem = 1024 + STAGES * kStageBytes + 2 * kBatch * kScaleBytes + 256;
    static_assert(BN * 512 <= STAGES * kStageBytes, "the parts meet where the tiles were");
    static_assert(BN % 16 == 0 && BN <= 128, "one chunk of scales");
    static_assert(2 * kBatch * kScaleBytes >= 4 * kStoreStage * 4, "staging of the stores");
};

__device__ __forceinline__ float cluster_ld(uint32_t at) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at));
    return x;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t at) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at));
    return x;
}

template <int BN, int STAGES>
__global__ void __launch_bounds__(kSplitThreads, 2) k_q8_matmul_split(const __grid_constant__ CUtensorMap map_p,
                                                                      const __grid_constant__ CUtensorMap map_q,
                                                                      const __grid_constant__ MmArgs a) {
    using S = SplitShape<BN, STAGES>;
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (su32(raw) & 1023)) & 1023);
    uint8_t* scale_sh = base + STAGES * S::kStageBytes;
    float* store_sh = reinterpret_cast<float*>(scale_sh);                        // once the products are done
    uint64_t* full = reinterpret_cast<uint64_t*>(scale_sh + 2 * kBatch * S::kScaleBytes);
    uint64_t* empty = full + STAGES;
    uint64_t* sfull = empty + STAGES;
    uint64_t* sempty = sfull + 2;
    uint64_t* done = sempty + 2;
    uint64_t* settled = done + 1;                // all that the products' warp issued is complete
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(settled + 1);
    uint32_t* gave_up = tmem_at + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull + i, 4);             // the scale warps
            mbar_init(sempty + i, 1);
        }
        mbar_init(done, 1);
        mbar_init(settled, 1);
        *gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    early_launch();
    if (warp == 0 && lane == 0) {
        prefetch_map(&map_p);
        prefetch_map(&map_q);
    }
    // Before the allocation: CTAs of two launches on one SM are the common case here, and one that allocates
    // while the other still runs slowed both (500 x 1000 x 5003: 14.6 us instead of 10.8).
    wait_for_predecessor();
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_at)),
                     "r"((uint32_t)S::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at, tmem_scales = tmem + BN;
    const int split = a.split, rank = blockIdx.x % split, tile = blockIdx.x / split;
    const int p0 = tile / a.tiles_q * 128, q0 = tile % a.tiles_q * BN;
    const int kb0 = (int)((int64_t)a.kblocks * rank / split), kbs = (int)((int64_t)a.kblocks * (rank + 1) / split) - kb0;
    const int groups = (kbs + 3) / 4;
    auto fail = [&] {
        atomicExch(gave_up, 1u);
        atomicCAS(a.error, 0u, ZS_DEVERR_MATMUL_WAIT);
    };

    if (warp == 0) {
        Ring ring;
        bool ok = true;
        for (int kb = 0; kb < kbs; ++kb) {
            if (ring.round > 0 && !(ok = warp_wait_or_look(empty + ring.at, ring.parity() ^ 1, a.wait_limit))) break;
            uint8_t* at = base + ring.at * S::kStageBytes;
            if (elect_one()) {
                mbar_expect_tx(full + ring.at, S::kStageBytes);
                tma_load(at, &map_p, (kb0 + kb) * 128, p0, full + ring.at);
                tma_load(at + 128 * 128, &map_q, (kb0 + kb) * 128, q0, full + ring.at);
            }
            __syncwarp();
            ring.next(STAGES);
        }
        if (!ok && lane == 0) fail();
        ring_settled(full, STAGES, ring.count(STAGES));      // no copy is under way when the CTA goes on
    } else if (warp == 1) {
        const uint32_t idesc = ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24);
        const uint64_t desc0 = operand_desc(su32(base)), sdesc0 = scales_desc(su32(scale_sh));
        bool ok = true;
        Ring ring, slots;
        // A group's scales overwrite those of four groups before: the products that read these are 13 blocks back
        // or more, and complete, since the ring's stages have been loaded again since.
        for (int kb = 0; kb < kbs; ++kb) {
            const int in = (kb >> 2) & (kBatch - 1);
            const uint32_t sfa = tmem_scales + in * S::kScaleCols;
            if ((kb & 3) == 0) {
                if (in == 0) {
                    if (!(ok = warp_wait(sfull + slots.at, slots.parity(), a.wait_limit))) break;
                    tc_fence_after();
                }
                const bool last = in == kBatch - 1 || kb + 4 >= kbs;
                if (elect_one()) {
                    const uint64_t from = sdesc0 + (((slots.at * kBatch + in) * S::kScaleBytes) >> 4);
                    tmem_copy_scales(sfa, from);
                    tmem_copy_scales(sfa + 4, from + (512 >> 4));
                    if (last) mma_commit(sempty + slots.at);
                }
                __syncwarp();
                if (last) slots.next(2);
            }
            if (!(ok = warp_wait(full + ring.at, ring.parity(), a.wait_limit))) break;
            tc_fence_after();
            const uint64_t da = desc0 + ((ring.at * S::kStageBytes) >> 4), db = da + ((128 * 128) >> 4);
            const uint32_t id = idesc | ((uint32_t)(kb & 3) << 29) | ((uint32_t)(kb & 3) << 4);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_scaled(tmem, da + 2 * k, db + 2 * k, id, sfa, sfa + 4, kb > 0 || k > 0);
                mma_commit(empty + ring.at);
            }
            __syncwarp();
            ring.next(STAGES);
        }
        if (!ok && lane == 0) fail();
        if (elect_one()) {
            if (ok) mma_commit(done);
            mma_commit(settled);
        }
        __syncwarp();
        // and neither a product nor an arrival
        ring_settled(empty, STAGES, ring.count(STAGES));
        ring_settled(sempty, 2, slots.count(2));
        ring_settled(done, 1, ok);
        ring_settled(settled, 1, 1);
    } else if (warp < 6) {
        // thread r of 128: P row r and Q row r of the tile (see the scale copy's layout below)
        Ring slots;
        bool ok = true;
        const int r = threadIdx.x - 64;
        uint8_t* mine = scale_sh + (r & 31) * 16 + (r >> 5) * 4;
        ScaleRow row[2];
        row[0].start(a.sp, a.ldsp, (int64_t)p0 + r, a.rows_p, kb0, kbs, a.kblocks);
        row[1].start(a.sq, a.ldsq, (int64_t)q0 + r, r < BN ? a.rows_q : 0, kb0, kbs, a.kblocks);
        for (int g = 0; g < groups; g += kBatch) {
            if (slots.round > 0 && !(ok = warp_wait_or_look(sempty + slots.at, slots.parity() ^ 1, a.wait_limit))) break;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t w[kBatch];
                row[c].take(w);
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    *reinterpret_cast<uint32_t*>(mine + (slots.at * kBatch + j) * S::kScaleBytes + c * 512) = w[j];
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull + slots.at);
            slots.next(2);
#pragma unroll
            for (int c = 0; c < 2; ++c) row[c].advance();
        }
        if (!ok && lane == 0) fail();
    } else {
        const int sub = warp & 3;
        const uint32_t from = tmem + ((uint32_t)(sub * 32) << 16);
        if (!warp_wait_or_look(done, 0, a.wait_limit)) {
            if (lane == 0) fail();
        } else {
            tc_fence_after();
            if (split == 1) {
                const int64_t p = (int64_t)p0 + sub * 32;                        // the warp's first row
                const int n = a.rows_q - q0, rows = a.rows_p - p < 32 ? (int)(a.rows_p - p) : 32;
#pragma unroll 1
                for (int c = 0; c < BN; c += 16) {
                    float f[16];
                    tmem_load16(from + c, f);
                    if (a.transposed) {
                        uint16_t* o = a.out + (int64_t)(q0 + c) * a.ldo + p + lane;
                        if (!a.first) {
                            uint16_t was[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) was[j] = c + j < n && lane < rows ? o[j * a.ldo] : 0;
#pragma unroll
                            for (int j = 0; j < 16; ++j) f[j] = fmaf(f[j], a.scale, bf16_to_f32(was[j]));
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) f[j] *= a.scale;
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c + j < n && lane < rows) o[j * a.ldo] = f32_to_bf16(f[j]);
                    } else {
                        store_rows16(a.out + p * a.ldo + q0 + c, a.ldo, f, rows, n - c, a.align, a.scale, a.first,
                                     store_sh + sub * kStoreStage);
                    }
                }
            } else {
                float* part = reinterpret_cast<float*>(base) + sub * 32 + lane;      // [column][128 rows]
#pragma unroll 1
                for (int c = 0; c < BN; c += 16) {
                    float f[16];
                    tmem_load16(from + c, f);
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c + j) * 128] = f[j];
                }
            }
            tc_fence_before();
        }
    }
    if (split > 1) {
        __syncthreads();
        cluster_sync();
        bool ok = true;
        for (int k = 0; k < split; ++k) {
            const uint32_t bad = cluster_ld_u32(at_rank(gave_up, k));        // all under way before the first is looked at
            ok = ok && bad == 0;
        }
        const int share = BN / split, c0 = rank * share, n = a.rows_q - q0;
        if (ok && a.transposed) {
            // four rows of a column per thread: they are neighbours in out
            for (int i = threadIdx.x; i < share * 32; i += kSplitThreads) {
                const int c = c0 + (i >> 5), r = (i & 31) * 4;
                const int64_t p = (int64_t)p0 + r;
                if (c >= n || p >= a.rows_p) continue;
                // every part's load under way before the first is added
                float4 x[kSplitMost];
#pragma unroll
                for (int k = 0; k < kSplitMost; ++k)
                    if (k < split) x[k] = cluster_ld4(at_rank(base + (c * 128 + r) * 4, k));
                float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < kSplitMost; ++k)
                    if (k < split) {
                        v[0] += x[k].x; v[1] += x[k].y; v[2] += x[k].z; v[3] += x[k].w;
                    }
                uint16_t* o = a.out + (int64_t)(q0 + c) * a.ldo + p;
                uint16_t was[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) was[j] = !a.first && p + j < a.rows_p ? o[j] : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = fmaf(v[j], a.scale, bf16_to_f32(was[j]));
                if (((uintptr_t)o & 7) == 0 && p + 4 <= a.rows_p) {
                    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (p + j < a.rows_p) o[j] = f32_to_bf16(v[j]);
                }
            }
        } else if (ok && share < 16) {
            for (int i = threadIdx.x; i < share * 128; i += kSplitThreads) {
                const int c = c0 + i % share, r = i / share;
                const int64_t p = (int64_t)p0 + r;
                if (c >= n || p >= a.rows_p) continue;
                float x[kSplitMost], v = 0.f;
#pragma unroll
                for (int k = 0; k < kSplitMost; ++k)
                    if (k < split) x[k] = cluster_ld(at_rank(base + (c * 128 + r) * 4, k));
#pragma unroll
                for (int k = 0; k < kSplitMost; ++k)
                    if (k < split) v += x[k];
                uint16_t* o = a.out + p * a.ldo + q0 + c;
                *o = f32_to_bf16(fmaf(v, a.scale, a.first ? 0.f : bf16_to_f32(*o)));
            }
        } else if (ok) {
            // 16 columns of a row per thread; the four warps that own staging memory
            if (warp >= 6) {
                const int r0 = (warp - 6) * 32;
                const int64_t p = (int64_t)p0 + r0;
                const int rows = a.rows_p - p < 32 ? (int)(a.rows_p - p) : 32;
                for (int c = c0; c < c0 + share; c += 16) {
                    float f[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) f[j] = 0.f;
#pragma unroll
                    for (int k = 0; k < kSplitMost; k += 2) {        // two parts' loads under way at a time
                        if (k >= split) break;
                        float x[2][16];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t at = at_rank(base + (c * 128 + r0 + lane) * 4, k + i);
#pragma unroll
                            for (int j = 0; j < 16; ++j) x[i][j] = cluster_ld(at + j * 512);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int j = 0; j < 16; ++j) f[j] += x[i][j];
                    }
                    store_rows16(a.out + p * a.ldo + q0 + c, a.ldo, f, rows, n - c, a.align, a.scale, a.first,
                                 store_sh + (warp - 6) * kStoreStage);
                }
            }
        }
        __syncwarp();
        cluster_sync();                          // no CTA leaves while another reads its part
    }
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)S::kTmemCols));
    }
}

// ------------------------------------------------------------------ large products: a persistent CTA pair per tile

// Tile of 256 P rows x BN Q rows per pair of CTAs.  Each CTA loads its 128 P rows and half of the Q rows
// (the tensor cores read the other half of Q from the other CTA), one thread of the leading CTA issues the
// products for both, and each CTA keeps 128 x BN fp32 accumulators in its own tensor memory.  The pairs are
// persistent and the accumulators doubled, so that eight warps write a tile out while the next one's
// products run; that and the scales leave BN at 224 or less.  Undoubled, a tile may have 256 columns: for
// products that every pair does in one tile.
constexpr int kPairThreads = 448;
constexpr int kPairStages = 6;
constexpr int kPairScaleBytes = 512 * 3;
constexpr int kPairSlots = 2;         // batches of scales in flight
constexpr int kPairTmemScales = 12;  // columns of one group's scales
constexpr int kScaleSets = 4;        // groups with columns of their own
template <int BN>
struct PairShape {
    static constexpr int kAccs = BN == 256 ? 1 : 2;
    static constexpr int kStageBytes = 128 * 128 + (BN / 2) * 128;
    static constexpr int kSmem = 1024 + kPairStages * kStageBytes + kPairSlots * kBatch * kPairScaleBytes + 8 * kStoreStage * 4 + 256;
    // kRowGroups: a table of the groups, their starts and the tiles before them
    static constexpr int table(int n_groups) { return (n_groups + 1) * 8; }
    static constexpr int kSmemMost = 227 * 1024;
    static_assert(kAccs * BN + kScaleSets * kPairTmemScales <= 512, "tensor memory");
    static_assert(BN % 32 == 0 && (BN / 2) % 16 == 0, "halves of whole 16-column loads");
};
constexpr int kPairGroup = 8;        // P tiles that share the same Q tiles at about the same time

// Products of groups in one launch, with the groups' places on the device: a group is an expert's rows.
//   kRowGroups  P's rows starts[g] .. starts[g + 1] times the group's own group_rows rows of Q
//   kFewRows    the same product with the operands' places exchanged: a tile is 256 of the group's own rows (of P now)
//               times as many of the starts' rows as there are, 32 to BN.  A block of the sum takes 180 + 0.48 N ns, so few
//               rows cost less as N than as 256 rows of P (37 tokens to 2 of 16 experts, 2048 x 4096: 27 us, 33 as 256 rows).
//   kSumGroups  the sum over columns starts[g] .. starts[g + 1] (multiples of 128) of both, one result per group
// Starts out of range are read as the nearest inside; with overlapping groups (more tiles than there can be) nothing is
// written, so that no tile lies outside.
enum { kNoGroups = 0, kRowGroups = 1, kSumGroups = 2, kFewRows = 3 };

// What the barriers of a pair's CTA have been or will be sent by copies and products, each to its ring in turn.  A CTA
// leaves only when all of it has arrived, after a wait that ran out as after the last tile: nothing may be under way
// when its shared and tensor memory go.
struct Sent {
    uint32_t loads;          // blocks that this CTA asked for
    uint32_t products;       // blocks multiplied
    uint32_t scales;         // batches of scales copied to tensor memory
    uint32_t sums;           // accumulators completed
};

// A pair's tile: its first rows of P and Q and where those that count end, its blocks of the sum, and its place in out.
struct Tile {
    int p0, q0, p_end, q_end;
    int width;                   // columns: BN, or fewer so that a group's are shared out evenly
    int kb0, kbs;
    int64_t out_row;             // row of out that P row 0 would have
    int out_col;                 // Q row that column 0 of out has
};
// Start g of the groups, in order and in range.
__device__ __forceinline__ int group_start(const MmArgs& a, int g, int most) {
    const int x = a.starts[g];
    return x < 0 ? 0 : x > most ? most : x;
}

template <int BN, int GROUPS>
__global__ void __launch_bounds__(kPairThreads, 1)
    k_q8_matmul_pair(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                     const __grid_constant__ CUtensorMap map_out, const __grid_constant__ MmArgs a) {
    constexpr int kStageBytes = PairShape<BN>::kStageBytes, kAccs = PairShape<BN>::kAccs;
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (su32(raw) & 1023)) & 1023);
    uint8_t* scale_sh = base + kPairStages * kStageBytes;
    float* store_sh = reinterpret_cast<float*>(scale_sh + kPairSlots * kBatch * kPairScaleBytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(store_sh + 8 * kStoreStage);   // leader: both CTAs' tiles landed
    uint64_t* empty = full + kPairStages;        // each CTA: the products have read the stage
    uint64_t* sfull = empty + kPairStages;       // leader: both CTAs' scales are in shared memory
    uint64_t* sempty = sfull + kPairSlots;       // each CTA: they are copied out
    uint64_t* done = sempty + kPairSlots;        // each CTA: an accumulator is complete
    uint64_t* acc_free = done + 2;               // leader: both CTAs have read it
    uint64_t* settled = acc_free + 2;            // each CTA: all that the products' warp issued is complete
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(settled + 1);
    uint32_t* gave_up = tmem_at + 1;             // set in both CTAs
    Sent* sent = reinterpret_cast<Sent*>(gave_up + 1);
    int* before = reinterpret_cast<int*>(store_sh + 8 * kStoreStage) + 64;       // kRowGroups: tiles before each group's,
    int* start = before + a.n_groups + 1;                                         // and its first row
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();        // CTA 0 of the pair leads
    constexpr uint16_t kBoth = 3;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < kPairSlots; ++i) {
            mbar_init(sfull + i, 8);             // the four scale warps of both CTAs
            mbar_init(sempty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(done + i, 1);
            mbar_init(acc_free + i, 16);         // the eight reading warps of both CTAs
        }
        mbar_init(settled, 1);
        *gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    early_launch();
    if (warp == 0 && lane == 0) {
        prefetch_map(&map_p);
        prefetch_map(&map_q);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_at)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    wait_for_predecessor();
    const uint32_t tmem = *tmem_at, tmem_scales = tmem + kAccs * BN;
    const int tiles_p = (int)(((int64_t)a.rows_p + 255) / 256);
    int64_t tiles = (int64_t)tiles_p * a.tiles_q;
    if constexpr (GROUPS == kSumGroups) tiles *= a.n_groups;
    if constexpr (GROUPS == kRowGroups || GROUPS == kFewRows) {
        // Tiles of the groups summed up: a thread adds a few neighbouring groups', the threads' sums are scanned.
        const int each = (a.n_groups + kPairThreads - 1) / kPairThreads, g0 = threadIdx.x * each;
        for (int g = threadIdx.x; g <= a.n_groups; g += kPairThreads) start[g] = group_start(a, g, GROUPS == kRowGroups ? a.rows_p : a.rows_q);
        __syncthreads();
        auto tiles_of = [&](int g) {
            const int lo = start[g], hi = start[g + 1];
            constexpr int kRows = GROUPS == kRowGroups ? 256 : BN;
            return hi > lo ? (int64_t)((hi - lo + kRows - 1) / kRows) * a.tiles_q : 0;
        };
        int64_t sum = 0;
        for (int g = g0; g < g0 + each && g < a.n_groups; ++g) sum += tiles_of(g);
        int64_t upto = sum;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int64_t x = __shfl_up_sync(~0u, upto, k);
            if (lane >= k) upto += x;
        }
        int64_t* warps = reinterpret_cast<int64_t*>(store_sh);
        if (lane == 31) warps[warp] = upto;
        __syncthreads();
        for (int w = 0; w < warp; ++w) upto += warps[w];
        int64_t at = upto - sum;
        for (int g = g0; g < g0 + each && g < a.n_groups; ++g) {
            before[g] = (int)at;
            at += tiles_of(g);
        }
        if (threadIdx.x == kPairThreads - 1) before[a.n_groups] = upto <= a.most_tiles ? (int)upto : 0;
        __syncthreads();
        tiles = before[a.n_groups];
    }
    const int64_t first_tile = blockIdx.x / 2, step = gridDim.x / 2;
    // Tile q of tiles_q over a group's columns: units of 32 shared out evenly, so that no tile computes columns that are not
    // there (2048 columns: two tiles in five of 224 columns and the others of 192, where ten of 224 compute 2240).
    const int all = GROUPS == kRowGroups ? a.group_rows : a.rows_q;
    const int units = (all + 31) / 32, few = units / a.tiles_q, wider = units - few * a.tiles_q;
    auto columns = [&](Tile& x, int q) {
        x.q0 = (q * few + (q < wider ? q : wider)) * 32;
        x.width = (few + (q < wider)) * 32;
    };
    // Tile `in` of `high` x tiles_q: kPairGroup P tiles at a time, within them Q tile by Q tile.
    auto strip = [&](int in, int high, int& p, int& q) {
        const int per = kPairGroup * a.tiles_q, s = in / per, rest = in - s * per;
        const int tall = high - s * kPairGroup < kPairGroup ? high - s * kPairGroup : kPairGroup;
        q = rest / tall;
        p = s * kPairGroup + rest - q * tall;
    };
    // the pair's tile t; g: the group of an earlier tile
    auto place = [&](int64_t t, int& g) {
        Tile x;
        int p, q;
        if constexpr (GROUPS == kRowGroups) {
            while (before[g + 1] <= (int)t) ++g;
            const int lo = start[g], hi = start[g + 1];
            strip((int)t - before[g], (hi - lo + 255) / 256, p, q);
            x = Tile{lo + p * 256, 0, hi, (g + 1) * a.group_rows, 0, 0, a.kblocks, 0, g * a.group_rows};
            columns(x, q);
            x.q0 += x.out_col;
        } else if constexpr (GROUPS == kFewRows) {
            while (before[g + 1] <= (int)t) ++g;
            const int in = (int)t - before[g];                                   // of tiles_q x ceil(rows / BN)
            q = in / a.tiles_q;
            p = in - q * a.tiles_q;
            x = Tile{g * a.group_rows + p * 256, start[g] + q * BN, (g + 1) * a.group_rows, start[g + 1], 0, 0, a.kblocks, 0, g * a.group_rows};
            x.width = x.q_end - x.q0 < BN ? (x.q_end - x.q0 + 31) / 32 * 32 : BN;
        } else if constexpr (GROUPS == kSumGroups) {
            const int per = tiles_p * a.tiles_q, most = a.kblocks * 128;
            g = (int)t / per;
            strip((int)t - g * per, tiles_p, p, q);
            const int lo = group_start(a, g, most), hi = group_start(a, g + 1, most);
            x = Tile{p * 256, 0, a.rows_p, a.rows_q, 0, lo / 128, 0, (int64_t)g * a.group_rows, 0};
            x.kbs = hi > lo ? (hi + 127) / 128 - x.kb0 : 0;
            columns(x, q);
        } else {
            const int64_t per = (int64_t)kPairGroup * a.tiles_q;
            const int s = (int)(t / per), in = (int)(t - s * per);
            const int width = tiles_p - s * kPairGroup < kPairGroup ? tiles_p - s * kPairGroup : kPairGroup;
            x = Tile{(s * kPairGroup + in % width) * 256, (in / width) * BN, a.rows_p, a.rows_q, BN, 0, a.kblocks, 0, 0};
        }
        return x;
    };
    auto fail = [&] {
        cluster_st(at_rank(gave_up, 0), 1);
        cluster_st(at_rank(gave_up, 1), 1);
        atomicCAS(a.error, 0u, ZS_DEVERR_MATMUL_WAIT);
    };

    if (warp == 0) {
        Ring ring;
        bool ok = true;
        int group = 0;
        const uint32_t full0 = at_rank(full, 0);
        for (int64_t t = first_tile; t < tiles && ok; t += step) {
            const Tile x = place(t, group);
            // where a group's rows end in the pair's first half, the second reads zeros past the matrix: not fetched, little power
            const int half = GROUPS == kNoGroups ? BN / 2 : x.width / 2, p = x.p0 + (int)rank * 128;
            const int row = (GROUPS == kRowGroups || GROUPS == kFewRows) && p >= x.p_end ? a.rows_p : p;
            for (int kb = x.kb0; kb < x.kb0 + x.kbs; ++kb) {
                if (ring.round > 0 && !(ok = warp_wait_or_look(empty + ring.at, ring.parity() ^ 1, a.wait_limit))) break;
                uint8_t* at = base + ring.at * kStageBytes;
                if (elect_one()) {
                    if (rank == 0) mbar_expect_tx(full + ring.at, 2 * kStageBytes);
                    tma_load_pair(at, &map_p, kb * 128, row, full0 + ring.at * 8);
                    tma_load_pair(at + 128 * 128, &map_q, kb * 128, x.q0 + (int)rank * half, full0 + ring.at * 8);
                }
                __syncwarp();
                ring.next(kPairStages);
            }
        }
        if (lane == 0) sent->loads = ring.count(kPairStages);
        if (!ok && lane == 0) fail();
    } else if (warp == 1 && rank == 0) {
        uint32_t idesc = ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((256u >> 4) << 24);
        const uint64_t desc0 = operand_desc(su32(base));
        const uint64_t sdesc0 = scales_desc(su32(scale_sh));
        bool ok = true;
        Ring ring, slots, acc, set;
        uint32_t sfa = tmem_scales;
        int group = 0;
        Tile here;
        if constexpr (GROUPS != kNoGroups) {
            if (first_tile < tiles) here = place(first_tile, group);
        }
        // A group's scales overwrite those of four groups before, whose products are complete: within a tile and into
        // the next they are nine blocks back or more, and the ring's six stages have been loaded again since; those
        // of the tile before that have been read out.
        for (int64_t t = first_tile; t < tiles && ok; t += step) {
            if (acc.round > 0 && !(ok = warp_wait_cluster(acc_free + acc.at, acc.parity() ^ 1, a.wait_limit))) break;
            tc_fence_after();
            const uint32_t sums = tmem + acc.at * BN;
            const int kbs = GROUPS == kNoGroups ? a.kblocks : here.kbs;
            if constexpr (GROUPS != kNoGroups) idesc = ((uint32_t)(here.width >> 3) << 17) | (1u << 23) | ((256u >> 4) << 24);
            for (int kb = 0; kb < kbs; ++kb) {
                if ((kb & 3) == 0) {
                    const int in = (kb >> 2) & (kBatch - 1);         // group of the batch
                    sfa = tmem_scales + set.at * kPairTmemScales;
                    set.next(kScaleSets);
                    if (in == 0) {
                        if (!(ok = warp_wait_cluster(sfull + slots.at, slots.parity(), a.wait_limit))) break;
                        tc_fence_after();
                    }
                    const bool last = in == kBatch - 1 || kb + 4 >= kbs;
                    if (elect_one()) {
                        const uint64_t from = sdesc0 + (((slots.at * kBatch + in) * kPairScaleBytes) >> 4);
                        tmem_copy_scales_pair(sfa, from);
                        tmem_copy_scales_pair(sfa + 4, from + (512 >> 4));
                        tmem_copy_scales_pair(sfa + 8, from + (1024 >> 4));
                        if (last) mma_commit_pair(sempty + slots.at, kBoth);
                    }
                    __syncwarp();
                    if (last) slots.next(kPairSlots);
                }
                if (!(ok = warp_wait(full + ring.at, ring.parity(), a.wait_limit))) break;
                tc_fence_after();
                const uint64_t da = desc0 + ((ring.at * kStageBytes) >> 4), db = da + ((128 * 128) >> 4);
                const uint32_t id = idesc | ((uint32_t)(kb & 3) << 29) | ((uint32_t)(kb & 3) << 4);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_scaled_pair(sums, da + 2 * k, db + 2 * k, id, sfa, sfa + 4, kb > 0 || k > 0);
                    mma_commit_pair(empty + ring.at, kBoth);
                }
                __syncwarp();
                ring.next(kPairStages);
            }
            if (!ok) break;
            if (elect_one()) mma_commit_pair(done + acc.at, kBoth);
            __syncwarp();
            acc.next(kAccs);
            if constexpr (GROUPS != kNoGroups) {
                if (t + step < tiles) here = place(t + step, group);             // while the last products run
            }
        }
        if (elect_one()) mma_commit_pair(settled, kBoth);
        __syncwarp();
        if (lane < 2) {
            cluster_st(at_rank(&sent->products, lane), ring.count(kPairStages));
            cluster_st(at_rank(&sent->scales, lane), slots.count(kPairSlots));
            cluster_st(at_rank(&sent->sums, lane), acc.count(kAccs));
        }
        if (!ok && lane == 0) fail();
    } else if (warp >= 2 && warp < 6) {
        // thread r of 128: P row r, Q rows r and 128 + r of the tile; the scale copy wants row r's word at
        // (r % 32) * 16 + (r / 32) * 4
        Ring slots;
        bool ok = true;
        const int r = threadIdx.x - 64;
        int group = 0;
        uint8_t* mine = scale_sh + (r & 31) * 16 + (r >> 5) * 4;
        for (int64_t t = first_tile; t < tiles && ok; t += step) {
            const Tile x = place(t, group);
            const int groups = (x.kbs + 3) / 4;
            ScaleRow row[3];
            row[0].start(a.sp, a.ldsp, (int64_t)x.p0 + rank * 128 + r, a.rows_p, x.kb0, x.kbs, a.kblocks);
            row[1].start(a.sq, a.ldsq, (int64_t)x.q0 + r, a.rows_q, x.kb0, x.kbs, a.kblocks);
            row[2].start(a.sq, a.ldsq, (int64_t)x.q0 + 128 + r, BN > 128 + r ? a.rows_q : 0, x.kb0, x.kbs, a.kblocks);
            for (int g = 0; g < groups; g += kBatch) {
                if (slots.round > 0 && !(ok = warp_wait_or_look(sempty + slots.at, slots.parity() ^ 1, a.wait_limit))) break;
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    uint32_t w[kBatch];
                    row[c].take(w);
#pragma unroll
                    for (int j = 0; j < kBatch; ++j)
                        *reinterpret_cast<uint32_t*>(mine + (slots.at * kBatch + j) * kPairScaleBytes + c * 512) = w[j];
                }
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
        Ring acc;
        int group = 0;
        for (int64_t t = first_tile; t < tiles; t += step, acc.next(kAccs)) {
            const Tile x = place(t, group);
            if (!warp_wait_or_look(done + acc.at, acc.parity(), a.wait_limit)) {
                if (lane == 0) fail();
                break;
            }
            tc_fence_after();
            if constexpr (GROUPS == kFewRows) {
                // lanes hold neighbouring columns of out, the accumulator's columns are its rows
                const int col = x.p0 - x.out_col + (int)rank * 128 + sub * 32 + lane;
                const uint32_t from = tmem + acc.at * BN + ((uint32_t)(sub * 32) << 16);
#pragma unroll 1
                for (int c = half * 32; c < x.width; c += 64) {
                    float f[32];
                    tmem_load32(from + c, f);
                    uint16_t* o = a.out + (int64_t)(x.q0 + c) * a.ldo + col;
                    const int rows = col < a.group_rows ? x.q_end - x.q0 - c : 0;
                    if (!a.first) {
                        uint16_t was[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) was[j] = j < rows ? o[j * a.ldo] : 0;
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = fmaf(f[j], a.scale, bf16_to_f32(was[j]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] *= a.scale;
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < rows) o[j * a.ldo] = f32_to_bf16(f[j]);
                }
            } else if constexpr (GROUPS != kNoGroups) {
                // Pieces of 32 columns, in turn for the two halves of the warps.  Whole pieces that are only written go by tiled
                // copies: 64 bytes of a row at once and nothing of the warp's time, where its own stores touch 32 lines for 32
                // bytes each (8 x 5504 x 2048 over 750 rows each, whose tiles are written about as fast as they are
                // computed: 82 us, 91 by the warps).
                const bool sum = GROUPS != kSumGroups || x.kbs > 0;              // the empty sum: zeros, or out as it is
                const int64_t p = (int64_t)x.p0 + rank * 128 + sub * 32;         // the warp's first row
                int rows = x.p_end - p < 32 ? (int)(x.p_end - p) : 32;
                if (!sum && !a.first) rows = 0;
                const bool whole_rows = a.tiled && rows == 32;
                const uint32_t from = tmem + acc.at * BN + ((uint32_t)(sub * 32) << 16);
                float* stage = store_sh + (warp - 6) * kStoreStage;
#pragma unroll 1
                for (int c = half * 32; c < x.width; c += 64) {
                    float f[32];
                    tmem_load32(from + c, f);
                    if (GROUPS == kSumGroups && !sum) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = 0.f;
                    }
                    if (lane == 0) tma_stores_read();                            // the piece before has left the staging
                    __syncwarp();
                    const int q = x.q0 - x.out_col + c, n = x.q_end - x.out_col - q;
                    // A group's last columns by the warps: a tiled store cut off inside 16 bytes writes all 16, and what lies
                    // between the rows is the caller's.
                    if (whole_rows && n >= 32) {
                        uint4* to = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(stage) + lane * 64);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(f[8 * k + 2 * j] * a.scale, f[8 * k + 2 * j + 1] * a.scale);
                            to[k ^ ((lane >> 1) & 3)] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) tma_store(&map_out, stage, q, (int)(x.out_row + p));
                    } else {
                        uint16_t* o = a.out + (x.out_row + p) * a.ldo + q;
                        store_rows16(o, a.ldo, reinterpret_cast<float(&)[16]>(f[0]), rows, n, a.align, a.scale, a.first, stage);
                        store_rows16(o + 16, a.ldo, reinterpret_cast<float(&)[16]>(f[16]), rows, n - 16, a.align, a.scale, a.first, stage);
                    }
                }
            } else {
                const int64_t p = (int64_t)x.p0 + rank * 128 + sub * 32;         // the warp's first row
                const int rows = x.p_end - p < 32 ? (int)(x.p_end - p) : 32;
                constexpr int kHalf = BN / 2;                                    // columns of one warp
                const int qh = x.q0 + half * kHalf;
                uint16_t* o = a.out + p * a.ldo + qh;
                const uint32_t from = tmem + acc.at * BN + half * kHalf + ((uint32_t)(sub * 32) << 16);
#pragma unroll 1
                for (int c = 0; c < kHalf; c += 16) {
                    float f[16];
                    tmem_load16(from + c, f);
                    store_rows16(o + c, a.ldo, f, rows, x.q_end - qh - c, a.align, a.scale, a.first,
                                 store_sh + (warp - 6) * kStoreStage);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(at_rank(acc_free + acc.at, 0));
        }
        if ((GROUPS == kRowGroups || GROUPS == kSumGroups) && lane == 0) tma_stores_done();
    }
    __syncthreads();
    cluster_sync();                              // nobody issues anything any more, and what was issued is known
    const bool bad = *gave_up != 0;
    if (warp == 0) {
        // Both CTAs' copies count on the leader's barriers, each phase of which wants a block of both.  CTAs that gave
        // up may have asked for different numbers of blocks (six apart at most: a stage is loaded again only when the
        // products have read it, which takes both): the leader makes the phases whole, and waits for them.
        if (bad && rank == 0) {
            const uint32_t mine = sent->loads, other = cluster_ld_u32(at_rank(&sent->loads, 1));
            if (lane == 0) {
                for (uint32_t j = other; j < mine; ++j) mbar_complete_tx(full + j % kPairStages, kStageBytes);
                for (uint32_t j = mine; j < other; ++j) mbar_expect_tx(full + j % kPairStages, kStageBytes);
            }
            __syncwarp();
            ring_settled(full, kPairStages, mine > other ? mine : other);
        }
        ring_settled(empty, kPairStages, sent->products);
        ring_settled(sempty, kPairSlots, sent->scales);
        ring_settled(done, kAccs, sent->sums);
        ring_settled(settled, 1, 1);
    }
    if (bad) {                                   // in both CTAs: the other's copies are counted here, tensor memory is both's
        __syncthreads();
        cluster_sync();
    }
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

// The two operands' tensor maps: boxes of 128 columns, swizzled as the products read them.
cudaError_t make_maps(CUtensorMap* mp, CUtensorMap* mq, const Q8& p, const Q8& q, const MmArgs& a, int64_t k, int box_p, int box_q) {
    const cudaError_t e = make_map(mp, p.codes, false, a.rows_p, k, p.ld, box_p, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    return e != cudaSuccess ? e : make_map(mq, q.codes, false, a.rows_q, k, q.ld, box_q, 128, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int BN, int STAGES>
cudaError_t launch_mm_split(const Q8& p, const Q8& q, int64_t k, MmArgs& a, cudaStream_t st) {
    using S = SplitShape<BN, STAGES>;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = ready_once(ready, (const void*)k_q8_matmul_split<BN, STAGES>, S::kSmem);
    if (e != cudaSuccess) return e;
    CUtensorMap mp, mq;
    e = make_maps(&mp, &mq, p, q, a, k, 128, BN);
    if (e != cudaSuccess) return e;
    a.tiles_q = (a.rows_q + BN - 1) / BN;
    const int64_t tiles = (int64_t)((a.rows_p + 127) / 128) * a.tiles_q;
    // Split while the CTAs still fit one per SM and keep at least five blocks each, or two per SM and ten:
    // joining the parts costs 2-4 us, which more CTAs do not earn back (1 x 22016 x 4096, 172 tiles: 17.8 us
    // unsplit, 22.5 and 31.7 in 2 and 8 parts; 1 x 4096 x 4096, 32 tiles: 11.4 unsplit, 6.3 in 4, 6.6 in 8;
    // 37 x 4096 x 11008: 13.8 in 4, 12.9 in 8).
    a.split = 1;
    const int64_t sms = q8_host::sm_count();
    while (a.split < kSplitMost &&
           ((tiles * a.split * 2 <= sms && a.kblocks >= a.split * 2 * 5) ||
            (tiles * a.split * 2 <= 2 * sms && a.kblocks >= a.split * 2 * 10)))
        a.split *= 2;
    if (tiles * a.split > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * a.split));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = dependent_launch() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, k_q8_matmul_split<BN, STAGES>, mp, mq, a);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

// CTA pairs that are resident at once.
int64_t resident_pairs() { return q8_host::sm_count() / 2; }

template <int BN, int GROUPS = kNoGroups>
cudaError_t launch_mm_pair(const Q8& p, const Q8& q, int64_t k, MmArgs& a, cudaStream_t st) {
    constexpr bool kTable = GROUPS == kRowGroups || GROUPS == kFewRows;
    const int smem = PairShape<BN>::kSmem + (kTable ? PairShape<BN>::table(a.n_groups) : 0);
    const auto kern = k_q8_matmul_pair<BN, GROUPS>;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = ready_once(ready, (const void*)kern, kTable ? PairShape<BN>::kSmemMost : smem);
    if (e != cudaSuccess) return e;
    CUtensorMap mp, mq, mo;
    e = make_maps(&mp, &mq, p, q, a, k, 128, BN / 2);
    if (e != cudaSuccess) return e;
    mo = mp;
    if ((GROUPS == kRowGroups || GROUPS == kSumGroups) && a.tiled) {
        const int64_t rows = GROUPS == kRowGroups ? a.rows_p : (int64_t)a.rows_p * a.n_groups, cols = GROUPS == kRowGroups ? a.group_rows : a.rows_q;
        e = make_map(&mo, a.out, true, rows, cols, a.ldo * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
        if (e != cudaSuccess) return e;
    }
    const int64_t high = ((int64_t)a.rows_p + 255) / 256;
    a.tiles_q = GROUPS == kFewRows ? (a.group_rows + 255) / 256 : ((GROUPS == kRowGroups ? a.group_rows : a.rows_q) + BN - 1) / BN;
    // at most: a group's last rows may be a tile of their own
    auto with_ends = [&](int64_t tiles, int64_t rows) { return tiles + (a.n_groups < rows ? a.n_groups : rows); };
    const int64_t most = GROUPS == kRowGroups ? with_ends(high, a.rows_p) : GROUPS == kFewRows ? with_ends(((int64_t)a.rows_q + BN - 1) / BN, a.rows_q)
                         : GROUPS == kSumGroups ? high * a.n_groups : high;
    const int64_t tiles = most * a.tiles_q, room = resident_pairs();
    if (GROUPS != kNoGroups) {
        if (tiles > 0x7fffffff - 2 * room) return cudaErrorInvalidConfiguration;
        a.most_tiles = (int)tiles;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < room ? tiles : room)));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = dependent_launch() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, mp, mq, mo, a);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

// The tile width with the least time in the busiest pair, for `tp` tiles of P: rounds of tiles times the time of one.  Measured per block of
// the sum, one to three rounds of 4096 to 16384 columns, ns for tiles of 128 / 160 / 192 / 224 / 256 columns: 243 251
// 266 284 302; where rows of codes are not 128 bytes apart, or a multiple, and each row of a box touches two lines,
// 296 322 349 370 395.  Writing a tile out, 2.5 us, is hidden by the next tile's products but for the last one (and
// for 256 columns).
int pair_width(int64_t tp, int64_t rows_q, double kblocks, bool lines, int widest = 256) {
    int best = 128;
    double least = 1e300;
    const int64_t room = resident_pairs();
    for (int bn : {256, 224, 192, 160, 128}) {
        if (bn > widest) continue;
        const int64_t rounds = (tp * ((rows_q + bn - 1) / bn) + room - 1) / room;
        const double block = lines ? 180 + 0.48 * bn : 200 + 0.765 * bn;
        const double cost = (double)rounds * kblocks * block + 2500.0 * (bn == 256 ? rounds : 1);
        if (cost < least) {
            least = cost;
            best = bn;
        }
    }
    return best;
}

// Rows of out for an expert, on average, up to which they are the narrow operand: the caller's matrix decides, as the rows in
// use are known on the device only (with align 128 it has more, and so few tokens run as P there).  Microseconds as such and
// as P for 16, 64, 96 and 128 rows each, align 1: 16 experts of 2048 x 4096 29 31 35 38 and 34 35 35 36; 64 of 2048 x 2048
// 48 54 57 62 and 58 59 62 65; 8 of 5504 x 2048 23 24 25 28 and 25 25 25 27.
constexpr int kFewAverage = 96;

// The products of groups, in the width of least time for groups of equal size (their sizes are on the device).
template <int GROUPS>
cudaError_t launch_mm_groups(const Q8& p, const Q8& q, int64_t k, MmArgs& a, int64_t rows_q, cudaStream_t st) {
    const bool lines = ((p.ld | q.ld) & 127) == 0;
    const int64_t n = a.n_groups;
    const bool room256 = GROUPS != kRowGroups || PairShape<256>::kSmem + PairShape<256>::table(a.n_groups) <= PairShape<256>::kSmemMost;
    const int64_t tp = GROUPS == kRowGroups ? n * ((a.rows_p / n + 255) / 256) : n * (((int64_t)a.rows_p + 255) / 256);
    switch (pair_width(tp, rows_q, GROUPS == kRowGroups ? a.kblocks : (double)a.kblocks / n, lines, room256 ? 256 : 224)) {
        case 256: return launch_mm_pair<256, GROUPS>(p, q, k, a, st);
        case 224: return launch_mm_pair<224, GROUPS>(p, q, k, a, st);
        case 192: return launch_mm_pair<192, GROUPS>(p, q, k, a, st);
        case 160: return launch_mm_pair<160, GROUPS>(p, q, k, a, st);
        default: return launch_mm_pair<128, GROUPS>(p, q, k, a, st);
    }
}

}  // namespace

}  // namespace zs

using namespace zs::q8_host;

namespace {

int output_align(const void* out, int64_t ldo) { return ((uintptr_t)out & 31) == 0 && (ldo & 15) == 0 ? 32 : wide(out, ldo) ? 16 : 0; }

// What the two products of groups share: `rows_q` rows of b, `out_rows` of out.
int group_args(const char* fn, const zs::Q8& qa, const zs::Q8& qb, const int32_t* starts, int32_t n_groups, int64_t m, int64_t rows_q,
               int64_t group_rows, int64_t n, int64_t k, int64_t out_rows, float scale, int32_t first, void* out, int64_t ldo, zs::MmArgs* g) {
    if (!starts) return fail(fn, "starts is NULL");
    if ((uintptr_t)starts & 3) return fail(fn, "starts is not 4-byte aligned");
    if (!std::isfinite(scale)) return fail(fn, "scale must be finite");
    ZS_Q8_TRY(check_bf16(fn, "out", out, ldo, out_rows, n));
    *g = zs::MmArgs{};
    g->sp = qa.scales;
    g->sq = qb.scales;
    g->ldsp = qa.lds;
    g->ldsq = qb.lds;
    g->rows_p = (int)m;
    g->rows_q = (int)rows_q;
    g->kblocks = (int)((k + 127) / 128);
    g->starts = starts;
    g->n_groups = n_groups;
    g->group_rows = (int)group_rows;
    g->out = (uint16_t*)out;
    g->ldo = ldo;
    g->align = output_align(out, ldo);
    g->scale = scale;
    g->first = first != 0;
    g->tiled = g->first && g->align && ldo * 2 < (int64_t(1) << 40);
    g->wait_limit = zs::wait_limit().load(std::memory_order_relaxed);
    return ZS_OK;
}

int check_groups(const char* fn, int32_t n_groups, int64_t m, int64_t n, int64_t k) {
    if (n_groups < 1 || n_groups > ZS_MAX_EXPERTS) return fail(fn, "n_experts out of range");
    ZS_Q8_TRY(check_dim(fn, "m", m, 0));
    ZS_Q8_TRY(check_dim(fn, "n", n, 0));
    return check_dim(fn, "k", k, 0);
}

}  // namespace

extern "C" int zs_q8_matmul_experts(const zs_q8* a, const zs_q8* b, const int32_t* starts, int32_t n_experts, int64_t m, int64_t n,
                                    int64_t k, float scale, int32_t first, void* out, int64_t ldo, void* stream) {
    static const char* fn = "zs_q8_matmul_experts";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::Q8 qa, qb;
    zs::MmArgs g;
    ZS_Q8_TRY(check_groups(fn, n_experts, m, n, k));
    if (k < 1) return fail(fn, "k out of range");
    ZS_Q8_TRY(check_dim(fn, "n_experts * n", n_experts * n, 0));
    ZS_Q8_TRY(check_q8(fn, "a", a, m, k, false, &qa));
    ZS_Q8_TRY(check_q8(fn, "b", b, n_experts * n, k, false, &qb));
    ZS_Q8_TRY(group_args(fn, qa, qb, starts, n_experts, m, n_experts * n, n, n, k, m, scale, first, out, ldo, &g));
    if (m == 0 || n == 0) return ZS_OK;
    ZS_Q8_TRY(cuda_status(fn, zs::error_word(&g.error)));
    if (m <= (int64_t)zs::kFewAverage * n_experts) {
        std::swap(g.sp, g.sq);
        std::swap(g.ldsp, g.ldsq);
        std::swap(g.rows_p, g.rows_q);
        return cuda_status(fn, zs::launch_mm_pair<128, zs::kFewRows>(qb, qa, k, g, (cudaStream_t)stream));
    }
    return cuda_status(fn, zs::launch_mm_groups<zs::kRowGroups>(qa, qb, k, g, n, (cudaStream_t)stream));
}

extern "C" int zs_q8_matmul_experts_grad(const zs_q8* a, const zs_q8* b, const int32_t* starts, int32_t n_experts, int64_t m, int64_t n,
                                         int64_t k, float scale, int32_t first, void* out, int64_t ldo, void* stream) {
    static const char* fn = "zs_q8_matmul_experts_grad";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::Q8 qa, qb;
    zs::MmArgs g;
    ZS_Q8_TRY(check_groups(fn, n_experts, m, n, k));
    ZS_Q8_TRY(check_dim(fn, "n_experts * m", n_experts * m, 0));
    ZS_Q8_TRY(check_q8(fn, "a", a, m, k, false, &qa));
    ZS_Q8_TRY(check_q8(fn, "b", b, n, k, false, &qb));
    ZS_Q8_TRY(group_args(fn, qa, qb, starts, n_experts, m, n, m, n, k, n_experts * m, scale, first, out, ldo, &g));
    if (m == 0 || n == 0) return ZS_OK;
    const cudaStream_t st = (cudaStream_t)stream;
    if (k == 0) {
        if (!first) return ZS_OK;
        const int64_t rows = n_experts * m, blocks = (rows * n + 255) / 256;
        return cuda_status(fn, zs::launch_kernel(zs::k_q8_empty_sum, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st,
                                                 (uint16_t*)out, ldo, rows, n));
    }
    ZS_Q8_TRY(cuda_status(fn, zs::error_word(&g.error)));
    return cuda_status(fn, zs::launch_mm_groups<zs::kSumGroups>(qa, qb, k, g, n, st));
}

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
    g.kblocks = (int)((k + 127) / 128);
    g.out = (uint16_t*)out;
    g.ldo = ldo;
    g.transposed = swap;
    g.align = output_align(out, ldo);
    g.scale = scale;
    g.first = first != 0;
    g.wait_limit = zs::wait_limit().load(std::memory_order_relaxed);
    ZS_Q8_TRY(cuda_status(fn, zs::error_word(&g.error)));
    // Up to 64 rows of b as well: the small kernel's narrow tiles (8192 x 8 x 4096: 10.6 us, and 13.3 in pairs of CTAs;
    // 8192 x 64 x 4096: 11.8 and 13.0; 50000 x 64 x 2048: 22.8 and 22.1).
    cudaError_t e;
    if (!swap && n > 64 && ((m + 255) / 256) * ((n + 255) / 256) >= 24) {
        switch (zs::pair_width((m + 255) / 256, n, g.kblocks, ((qa.ld | qb.ld) & 127) == 0)) {
            case 256: e = zs::launch_mm_pair<256>(p, q, k, g, st); break;
            case 224: e = zs::launch_mm_pair<224>(p, q, k, g, st); break;
            case 192: e = zs::launch_mm_pair<192>(p, q, k, g, st); break;
            case 160: e = zs::launch_mm_pair<160>(p, q, k, g, st); break;
            default: e = zs::launch_mm_pair<128>(p, q, k, g, st); break;
        }
    } else if (g.rows_q <= 16) {
        e = zs::launch_mm_split<16, 5>(p, q, k, g, st);
    } else if (g.rows_q <= 32) {
        e = zs::launch_mm_split<32, 4>(p, q, k, g, st);
    } else if (g.rows_q <= 64) {
        e = zs::launch_mm_split<64, 4>(p, q, k, g, st);
    } else {
        e = zs::launch_mm_split<128, 3>(p, q, k, g, st);
    }
    return cuda_status(fn, e);
}
