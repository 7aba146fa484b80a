// Tokens to their experts' rows and back: sorted by expert, written there in 8 bits (or bf16), and brought back
// weighted, with the gradients.  All of it moves bytes: a token's row is read once however many experts it goes to, and
// an expert's row once.
#include "q8_rows.cuh"

namespace zs {

namespace {

// ------------------------------------------------------------------ sorting

// A stable counting sort in one launch.  The pairs (token, choice) are cut into segments, one per warp of a cluster's
// CTAs.  First pass: a warp counts its segment's pairs per expert, 32 at a time: lanes of equal experts find each other by
// one vote per bit of the expert, and one of them adds their number.  The counters are summed over the warps, and over
// the cluster's CTAs through distributed shared memory; the second pass goes through the segment again, with what the
// first found where it fits in registers, and gives each pair its place.  A counter has one writer at a time and the order
// of the pairs is kept: the same rows every time, without a workspace.  131072 pairs of 64 experts: 7.3 us; in eight
// CTAs 11.4, 12.5 with atomics for the counts, 28.7 with the match instruction, which takes its time once per different
// value.  What bounds it is the issue of the votes and counts on the cluster's SMs.
constexpr int kSortWarps = 32;

struct SortArgs {
    const void* ids;
    int n, experts, align;
    int seg;                         // pairs per warp, a multiple of 32
    int *row_of, *starts, *counts;
};

template <typename ID, int BATCH>
__global__ void __launch_bounds__(kSortWarps * 32) k_expert_sort(const __grid_constant__ SortArgs a) {
    extern __shared__ int sort_sh[];
    const int E = a.experts;
    int* hist = sort_sh;                         // [warp][expert]
    int* total = hist + kSortWarps * E;          // this CTA's pairs per expert (read by the whole cluster)
    int* first = total + E;                      // where this CTA's pairs of an expert go
    __shared__ int scan[kSortWarps];
    uint32_t rank, ctas;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kSortWarps * E; i += blockDim.x) hist[i] = 0;
    dependent_launch_prologue();
    __syncthreads();
    const int64_t lo = (int64_t)(rank * kSortWarps + warp) * a.seg;
    const int64_t hi = lo + a.seg < a.n ? lo + a.seg : a.n;
    const ID* ids = static_cast<const ID*>(a.ids);
    int* mine = hist + warp * E;
    // A batch of the segment: each lane's experts (-1: none) and the lanes with the same one.
    const int bits = 32 - __clz(E - 1);
    int id[BATCH];
    uint32_t same[BATCH];
    auto read = [&](int64_t base) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int64_t i = base + 32 * j + lane;
            const ID x = i < hi ? ids[i] : (ID)-1;
            id[j] = x >= 0 && x < (ID)E ? (int)x : -1;
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) same[j] = __ballot_sync(~0u, id[j] >= 0);
        for (int b = 0; b < bits; ++b)
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const uint32_t set = __ballot_sync(~0u, id[j] >> b & 1);
                same[j] &= id[j] >> b & 1 ? set : ~set;
            }
    };
    for (int64_t base = lo; base < hi; base += 32 * BATCH) {
        read(base);
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (id[j] >= 0 && lane == __ffs(same[j]) - 1) mine[id[j]] += __popc(same[j]);
            __syncwarp();
        }
    }
    __syncthreads();
    const int e = threadIdx.x;                   // at most as many experts as threads
    if (e < E) {
        int sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const int x = hist[w * E + e];
            hist[w * E + e] = sum;
            sum += x;
        }
        total[e] = sum;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    int before = 0, all = 0;
    if (e < E) {
        for (uint32_t c = 0; c < ctas; ++c) {
            uint32_t at;
            int x;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(su32(total + e)), "r"(c));
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
            before += c < rank ? x : 0;
            all += x;
        }
    }
    const int padded = (all + a.align - 1) / a.align * a.align;
    int upto = padded;                           // sum over the experts up to this one
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int x = __shfl_up_sync(~0u, upto, k);
        if (lane >= k) upto += x;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        int x = scan[lane];
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int y = __shfl_up_sync(~0u, x, k);
            if (lane >= k) x += y;
        }
        scan[lane] = x;
    }
    __syncthreads();
    if (warp > 0) upto += scan[warp - 1];
    if (e < E) {
        first[e] = upto - padded + before;
        if (rank == 0) {
            a.starts[e] = upto - padded;
            a.counts[e] = all;
            if (e == E - 1) a.starts[E] = upto;
        }
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");       // the other CTAs' totals are read
    for (int64_t base = lo; base < hi; base += 32 * BATCH) {
        if (hi - lo > 32 * BATCH) read(base);
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int64_t i = base + 32 * j + lane;
            const int at = id[j] >= 0 ? mine[id[j]] : 0;
            __syncwarp();
            if (id[j] >= 0 && lane == __ffs(same[j]) - 1) mine[id[j]] = at + __popc(same[j]);
            if (i < hi) a.row_of[i] = id[j] >= 0 ? first[id[j]] + at + __popc(same[j] & ((1u << lane) - 1)) : -1;
            __syncwarp();
        }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");         // nobody reads this CTA's any more
}

// ------------------------------------------------------------------ to the experts

// Rows [starts[e] + counts[e], starts[e + 1]) hold no token: zeros, for a later sum over an expert's rows.  pad_warps
// warps share an expert's.

struct Rows {
    const int *row_of, *starts, *counts;
    int64_t tokens, rows, cols;
    int choices, experts, chunks;    // chunks of 512 columns
    int pad_warps;
    Q8 y;                            // either may be missing
    uint16_t* y16;
    int64_t ldy16;
};

template <bool WIDE>
__device__ __forceinline__ void zero_padding(const Rows& a, int64_t warp, int64_t warps) {
    const int lane = threadIdx.x & 31;
    const V16 zero = {};
    for (int64_t u = warp; u < (int64_t)a.experts * a.pad_warps; u += warps) {
        const int e = (int)(u / a.pad_warps);
        int64_t lo = (int64_t)a.starts[e] + a.counts[e], hi = a.starts[e + 1];
        if (lo < 0) lo = 0;
        if (hi > a.rows) hi = a.rows;
        for (int64_t r = lo + u % a.pad_warps; r < hi; r += a.pad_warps)
            for (int64_t c = lane * 16; c - lane * 16 < a.cols; c += 512) {
                if (a.y.codes) store_code16(make_uint4(0, 0, 0, 0), 0, a.cols - c, a.y, r, c);
                if (a.y16) store16<WIDE>(a.y16 + r * a.ldy16 + c, zero, a.cols - c);
            }
    }
}

// The row of choice j of a token, from the lane that holds it; -1 where there is none inside the matrix.
__device__ __forceinline__ int64_t row_at(int held, int j, int64_t rows) {
    const int r = __shfl_sync(~0u, held, j);
    return r >= 0 && r < rows ? r : -1;
}

struct DispatchArgs {
    Rows r;
    const uint16_t* x;
    int64_t ldx;
};

// A warp takes 512 columns of a token: read, encoded once, and written to every row that the token goes to.  Bound by the
// bytes: 16384 x 2048 to 8 of 64 experts 54 us (338 MB, 50 at the copy rate), and 60 with a fixed share for each CTA.
template <bool WIDE>
__global__ void __launch_bounds__(256) k_expert_dispatch(const __grid_constant__ DispatchArgs a) {
    dependent_launch_prologue();
    const int64_t warp = gtid() >> 5, warps = gstride() >> 5;
    const int lane = threadIdx.x & 31;
    const Span sx = span_of(a.x, a.ldx, a.r.tokens, a.r.cols);
    for (int64_t u = warp; u < a.r.tokens * a.r.chunks; u += warps) {
        const int64_t t = u / a.r.chunks, c = (u - t * a.r.chunks) * 512 + lane * 16, n = a.r.cols - c;
        const V16 v = load16<WIDE>(a.x + t * a.ldx + c, n, sx);
        const int held = lane < a.r.choices ? a.r.row_of[t * a.r.choices + lane] : -1;
        uint32_t byte = 0;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (a.r.y.codes) {
            float2 f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = pair_of(v.w[i]);
            w = code16(f, byte);
        }
        for (int j = 0; j < a.r.choices; ++j) {
            const int64_t row = row_at(held, j, a.r.rows);
            if (row < 0) continue;
            if (a.r.y.codes) store_code16(w, byte, n, a.r.y, row, c);
            if (a.r.y16) store16<WIDE>(a.r.y16 + row * a.r.ldy16 + c, v, n);
        }
    }
    zero_padding<WIDE>(a.r, warp, warps);
}

// ------------------------------------------------------------------ back to the tokens

constexpr int kAtOnce = 4;           // rows of a token read at once


struct CombineArgs {
    const uint16_t *y, *residual;
    int64_t ldy, ldr, ldo, rows, cols, tokens;
    const int* row_of;
    const float* weights;            // nullptr: 1
    int choices, chunks;
    uint16_t* out;
};

// A warp takes 512 columns of a token: residual + sum of weight * row in the order of the choices, in fp32.  Bound by the
// bytes, four rows of a token on their way at once: 16384 x 2048 from 8 experts 91 us (605 MB, 89 at the copy rate).  With
// registers for 32 warps per SM in the place of 24, and some of them spilled, 118.
template <bool WIDE>
__global__ void __launch_bounds__(256) k_expert_combine(const __grid_constant__ CombineArgs a) {
    dependent_launch_prologue();
    const int64_t warp = gtid() >> 5, warps = gstride() >> 5;
    const int lane = threadIdx.x & 31;
    const Span sy = span_of(a.y, a.ldy, a.rows, a.cols), sr = span_of(a.residual, a.ldr, a.tokens, a.cols);
    for (int64_t u = warp; u < a.tokens * a.chunks; u += warps) {
        const int64_t t = u / a.chunks, c = (u - t * a.chunks) * 512 + lane * 16, n = a.cols - c;
        const int held = lane < a.choices ? a.row_of[t * a.choices + lane] : -1;
        const float weight = a.weights && lane < a.choices ? a.weights[t * a.choices + lane] : 1.f;
        float2 f[8];
        V16 v = {};
        if (a.residual) v = load16<WIDE>(a.residual + t * a.ldr + c, n, sr);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = pair_of(v.w[i]);
        for (int j0 = 0; j0 < a.choices; j0 += kAtOnce) {
            V16 y[kAtOnce];
            bool live[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int64_t row = j0 + j < a.choices ? row_at(held, j0 + j, a.rows) : -1;
                live[j] = row >= 0;
                if (live[j]) y[j] = load16<WIDE>(a.y + row * a.ldy + c, n, sy);
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const float w = __shfl_sync(~0u, weight, (j0 + j) & 31);
                if (!live[j]) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = q8_fma2(pair_of(y[j].w[i]), make_float2(w, w), f[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v.w[i] = pack_bf16x2(f[i].x, f[i].y);
        store16<WIDE>(a.out + t * a.ldo + c, v, n);
    }
}

struct CombineBackArgs {
    Rows r;
    const uint16_t *dout, *y;
    int64_t lddout, ldy;
    const float* weights;            // nullptr: 1
    float* dweights;                 // nullptr: not wanted
};

constexpr int kMaxChoices = ZS_MAX_CHOICES;
constexpr int kBackWarps = 8;        // at most, per token
constexpr int kBackCtas = 4;         // resident (with rows in registers 149 us; 169 and 187 with 3 and 5)

// 16 columns of 8 neighbouring lanes, times w, in the format.  `top` is the block's largest finite magnitude before w:
// |w| times it is the largest after (rounding keeps the order), and w and the block's inverse scale are one factor where
// that is exact: where no value that matters comes near the ends of fp32's range (usual: top is in 2^-100 .. 2^100).
__device__ __forceinline__ uint4 code16_scaled(const float2 (&f)[8], float w, float top, bool usual, uint32_t& byte) {
    const float most = top * fabsf(w);           // and so |w| is above 2^-200 and below 2^228
    if (!__all_sync(~0u, most >= 0x1p-100f && most < __int_as_float(0x7f800000) && usual)) {
        float2 g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = q8_mul2(f[i], make_float2(w, w));
        return code16(g, byte);
    }
    byte = q8_scale_byte(most);
    const float by = w * q8_inverse(byte);
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 a = q8_mul2(f[2 * k], make_float2(by, by)), b = q8_mul2(f[2 * k + 1], make_float2(by, by));
        q[k] = q8_pack4(a.x, a.y, b.x, b.y);
    }
    return make_uint4(q[0], q[1], q[2], q[3]);
}

// A CTA takes a token, a warp of it 512 columns at a time: the gradient row stays in registers, and the experts' next rows
// are on their way to shared memory, to each lane's own places in it, while one is worked on.  What bounds it is how much
// is on its way: 16384 x 2048 with 8 choices takes 133 us (its 876 MB 129 at the copy rate) with three rows or four, 160 with
// six, for which fewer CTAs fit an SM, and took 150 with the next row in registers.
template <bool WIDE>
constexpr int kBackSlot = WIDE ? 32 : kSlot;             // bytes of a lane's 16 columns
constexpr int kBackRows = 3;                             // rows under way, the one worked on among them
template <bool WIDE>
__global__ void __launch_bounds__(32 * kBackWarps, kBackCtas) k_expert_combine_backward(const __grid_constant__ CombineBackArgs a) {
    __shared__ float dots[kBackWarps][kMaxChoices];
    extern __shared__ __align__(16) uint8_t back_sh[];   // [warp][row][lane]
    dependent_launch_prologue();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = blockDim.x >> 5;
    uint8_t* slots = back_sh + (warp * kBackRows * 32 + lane) * kBackSlot<WIDE>;
    const Span sd = span_of(a.dout, a.lddout, a.r.tokens, a.r.cols), sy = span_of(a.y, a.ldy, a.r.rows, a.r.cols);
    const int K = a.r.choices;
    const int64_t t = blockIdx.x;
    if (t < a.r.tokens) {
        const int held = lane < K ? a.r.row_of[t * K + lane] : -1;
        const float weight = a.weights && lane < K ? a.weights[t * K + lane] : 1.f;
        float dot = 0.f;                         // of choice `lane`
        for (int ch = warp; ch < a.r.chunks; ch += group) {
            const int64_t c = (int64_t)ch * 512 + lane * 16, n = a.r.cols - c;
            const V16 d = load16<WIDE>(a.dout + t * a.lddout + c, n, sd);
            auto slot = [&](int j) { return slots + j % kBackRows * (32 * kBackSlot<WIDE>); };
            auto fetch = [&](int j) {
                const int64_t row = j < K ? row_at(held, j & 31, a.r.rows) : -1;
                if (a.dweights && row >= 0) {
                    const uint16_t* from = a.y + row * a.ldy + c;
                    if (WIDE) {
                        if (n >= 8) async16(slot(j), reinterpret_cast<const uint8_t*>(from), 16);
                        else if (n > 0) async16(slot(j), reinterpret_cast<const uint8_t*>(from), (int)n * 2);
                        if (n >= 16) async16(slot(j) + 16, reinterpret_cast<const uint8_t*>(from + 8), 16);
                        else if (n > 8) async16(slot(j) + 16, reinterpret_cast<const uint8_t*>(from + 8), (int)(n - 8) * 2);
                    } else {
                        fetch16(slot(j), from, n, sy);
                    }
                }
                async_commit();
            };
#pragma unroll
            for (int j = 0; j < kBackRows - 1; ++j) fetch(j);
            float2 f[8];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] = pair_of(d.w[i]);
                top = q8_top2(top, f[i]);
            }
#pragma unroll
            for (int k = 1; k < 8; k <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
            const bool usual = top >= 0x1p-100f && top <= 0x1p100f;
#pragma unroll 1
            for (int j = 0; j < K; ++j) {
                fetch(j + kBackRows - 1);
                const int64_t row = row_at(held, j, a.r.rows);
                const float w = __shfl_sync(~0u, weight, j);
                asm volatile("cp.async.wait_group %0;" ::"n"(kBackRows - 1) : "memory");
                if (row < 0) continue;
                if (a.r.y.codes) {
                    uint32_t byte;
                    const uint4 x = code16_scaled(f, w, top, usual, byte);
                    store_code16(x, byte, n, a.r.y, row, c);
                }
                if (a.r.y16) {
                    V16 v;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v.w[i] = pack_bf16x2(f[i].x * w, f[i].y * w);
                    store16<WIDE>(a.r.y16 + row * a.r.ldy16 + c, v, n);
                }
                if (a.dweights) {
                    float sum = 0.f;
                    if (n > 0) {                 // elsewhere nothing was read
                        V16 y;
                        if (WIDE) {
                            const uint4 x0 = reinterpret_cast<const uint4*>(slot(j))[0], x1 = reinterpret_cast<const uint4*>(slot(j))[1];
                            y = V16{{x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w}};
                            if (n <= 8) y.w[4] = y.w[5] = y.w[6] = y.w[7] = 0;
                        } else {
                            y = take16(slot(j), a.y + row * a.ldy + c, n);
                        }
                        float2 s = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) s = q8_fma2(f[i], pair_of(y.w[i]), s);
                        sum = s.x + s.y;
                    }
#pragma unroll
                    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(~0u, sum, k);
                    if (lane == j) dot += sum;
                }
            }
        }
        if (a.dweights) {
            if (lane < K) dots[warp][lane] = dot;
            __syncthreads();
            if (threadIdx.x < K) {
                float sum = 0.f;
                for (int w = 0; w < group; ++w) sum += dots[w][threadIdx.x];
                a.dweights[t * K + threadIdx.x] = sum;
            }
        }
    }
    zero_padding<WIDE>(a.r, gtid() >> 5, gstride() >> 5);
}

// ------------------------------------------------------------------ host

using q8_host::fail;

int check_ints(const char* fn, const char* name, const void* p, bool needed) {
    if (!p && needed) return fail(fn, std::string(name) + " is NULL");
    if ((uintptr_t)p & 3) return fail(fn, std::string(name) + " is not 4-byte aligned");
    return ZS_OK;
}

int check_routes(const char* fn, int64_t tokens, int32_t choices, int32_t experts) {
    ZS_Q8_TRY(q8_host::check_dim(fn, "tokens", tokens, 0));
    if (choices < 1 || choices > ZS_MAX_CHOICES) return fail(fn, "choices out of range");
    if (experts < 1 || experts > ZS_MAX_EXPERTS) return fail(fn, "n_experts out of range");
    return ZS_OK;
}

// CTAs of the sort's cluster: one up to 1024 pairs (3.2 us; 4096 pairs take 4.8 in one and 3.5 in eight), eight, and sixteen
// past 65536 (131072: 7.3 us; 11.4 in eight) where the device has room for such clusters.
constexpr int kSortOne = 1024, kSortEight = 65536;

template <typename ID, int BATCH>
cudaError_t launch_sort(const SortArgs& a, int ctas, cudaStream_t st) {
    constexpr int per = (kSortWarps + 2) * 4;
    static std::atomic<uint64_t> ready{0};
    const auto kern = k_expert_sort<ID, BATCH>;
    cudaError_t e = ready_once(ready, (const void*)kern, per * ZS_MAX_EXPERTS);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kSortWarps * 32);
    cfg.dynamicSmemBytes = per * ZS_MAX_EXPERTS;         // what the occupancy is asked for
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = dependent_launch() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (ctas > 8) {                              // past the portable size: asked for once per device
        static std::atomic<uint64_t> asked{0}, fits{0};
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        const uint64_t bit = dev < kMaxDevices ? uint64_t(1) << dev : 0;
        if (!(asked.load(std::memory_order_acquire) & bit)) {
            int clusters = 0;
            if (cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess && clusters > 0)
                fits.fetch_or(bit, std::memory_order_release);
            cudaGetLastError();
            asked.fetch_or(bit, std::memory_order_release);
        }
        if (!(fits.load(std::memory_order_acquire) & bit)) return cudaErrorNotSupported;
    }
    cfg.dynamicSmemBytes = per * a.experts;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

// The sort with `ctas` CTAs: each warp's part of the pairs, and as many ids at once as it has (16 at once for a part of
// eight cost as much as for sixteen: 65536 pairs 11.0 us and 6.9).
template <typename ID>
cudaError_t launch_sort(SortArgs a, int ctas, cudaStream_t st) {
    const int64_t per = (int64_t)ctas * kSortWarps * 32;
    a.seg = (int)((a.n + per - 1) / per * 32);
    return a.seg <= 32    ? launch_sort<ID, 1>(a, ctas, st)
           : a.seg <= 128 ? launch_sort<ID, 4>(a, ctas, st)
           : a.seg <= 256 ? launch_sort<ID, 8>(a, ctas, st)
                          : launch_sort<ID, 16>(a, ctas, st);
}
template <typename ID>
cudaError_t launch_sort(const SortArgs& a, cudaStream_t st) {
    if (a.n > kSortEight) {
        const cudaError_t e = launch_sort<ID>(a, 16, st);
        if (e != cudaErrorNotSupported) return e;
    }
    return launch_sort<ID>(a, a.n <= kSortOne ? 1 : 8, st);
}

template <bool WIDE>
cudaError_t launch_back(const CombineBackArgs& a, unsigned ctas, int group, cudaStream_t st) {
    constexpr int per = kBackRows * 32 * kBackSlot<WIDE>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = ready_once(ready, (const void*)k_expert_combine_backward<WIDE>, per * kBackWarps);
    if (e != cudaSuccess) return e;
    return launch_kernel(k_expert_combine_backward<WIDE>, dim3(ctas), dim3(32 * group), a.dweights ? per * group : 0, st, a);
}

// CTAs for `warps` warps of work, `per` to a CTA, each with work of its own: CTAs that end make room for the next, so the
// work goes to the SMs as they get through it.  Past 2^31 CTAs the kernels go round.
unsigned grid_for(int64_t warps, int per) {
    const int64_t ctas = (warps + per - 1) / per, most = 0x7fffffff;
    return (unsigned)(ctas < 1 ? 1 : ctas < most ? ctas : most);
}

}  // namespace

}  // namespace zs

using namespace zs::q8_host;

extern "C" int zs_expert_sort(const void* ids, int32_t id_bytes, int64_t tokens, int32_t choices, int32_t n_experts, int32_t align,
                              int32_t* row_of, int32_t* starts, int32_t* counts, void* stream) {
    static const char* fn = "zs_expert_sort";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    ZS_Q8_TRY(zs::check_routes(fn, tokens, choices, n_experts));
    if (id_bytes != 4 && id_bytes != 8) return fail(fn, "id_bytes must be 4 or 8");
    const int64_t n = tokens * choices;
    if (align < 1 || align > ZS_MAX_EXPERT_ALIGN) return fail(fn, "align out of range");
    if (n + (int64_t)n_experts * (align - 1) > kMaxDim) return fail(fn, "the experts' rows pass 2^31 - 256");
    if (!ids && n > 0) return fail(fn, "ids is NULL");
    if ((uintptr_t)ids & (id_bytes - 1)) return fail(fn, "ids is not aligned to its elements");
    ZS_Q8_TRY(zs::check_ints(fn, "row_of", row_of, n > 0));
    ZS_Q8_TRY(zs::check_ints(fn, "starts", starts, true));
    ZS_Q8_TRY(zs::check_ints(fn, "counts", counts, true));
    zs::SortArgs a{ids, (int)n, n_experts, align, 0, row_of, starts, counts};
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = id_bytes == 4 ? zs::launch_sort<int32_t>(a, st) : zs::launch_sort<int64_t>(a, st);
    return cuda_status(fn, e);
}

namespace {

// The places of the experts' rows and what goes there, as zs_expert_dispatch and zs_expert_combine_backward take them.
int check_rows(const char* fn, const char* q_name, const char* b_name, const int32_t* row_of, int64_t tokens, int32_t choices,
               const int32_t* starts, const int32_t* counts, int32_t n_experts, int64_t rows, int64_t cols, const zs_q8* q, void* b,
               int64_t ldb, zs::Rows* out) {
    ZS_Q8_TRY(zs::check_routes(fn, tokens, choices, n_experts));
    ZS_Q8_TRY(check_dim(fn, "rows", rows, 0));
    ZS_Q8_TRY(check_dim(fn, "cols", cols, 1));
    ZS_Q8_TRY(zs::check_ints(fn, "row_of", row_of, tokens > 0));
    ZS_Q8_TRY(zs::check_ints(fn, "starts", starts, true));
    ZS_Q8_TRY(zs::check_ints(fn, "counts", counts, true));
    *out = zs::Rows{row_of, starts, counts, tokens, rows, cols, choices, n_experts, (int)((cols + 511) / 512), 1, {}, (uint16_t*)b, ldb};
    // an expert's rows without a token: about half of what `rows` has beyond the choices, if all are kept
    const int64_t beyond = (rows - tokens * choices) / n_experts;
    out->pad_warps = beyond < 4 ? 4 : beyond < 128 ? (int)beyond : 128;
    ZS_Q8_TRY(check_q8(fn, q_name, q, rows, cols, true, &out->y));
    if (b) ZS_Q8_TRY(check_bf16(fn, b_name, b, ldb, rows, cols));
    return ZS_OK;
}

}  // namespace

extern "C" int zs_expert_dispatch(const void* x, int64_t ldx, int64_t tokens, int64_t cols, const int32_t* row_of, int32_t choices,
                                  const int32_t* starts, const int32_t* counts, int32_t n_experts, int64_t rows, const zs_q8* y,
                                  void* y_bf16, int64_t ldy, void* stream) {
    static const char* fn = "zs_expert_dispatch";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::DispatchArgs a{};
    ZS_Q8_TRY(check_rows(fn, "y", "y_bf16", row_of, tokens, choices, starts, counts, n_experts, rows, cols, y, y_bf16, ldy, &a.r));
    ZS_Q8_TRY(check_bf16(fn, "x", x, ldx, tokens, cols));
    if (!y && !y_bf16) return fail(fn, "y and y_bf16 are both NULL");
    if (tokens == 0 || rows == 0) return ZS_OK;
    a.x = (const uint16_t*)x;
    a.ldx = ldx;
    const bool w = wide(x, ldx, 32) && (!y_bf16 || wide(y_bf16, ldy, 32));
    int64_t work = tokens * a.r.chunks;
    if (work < (int64_t)n_experts * a.r.pad_warps) work = (int64_t)n_experts * a.r.pad_warps;
    return cuda_status(fn, zs::launch_kernel(w ? zs::k_expert_dispatch<true> : zs::k_expert_dispatch<false>,
                                             dim3(zs::grid_for(work, 8)), dim3(256), 0, (cudaStream_t)stream, a));
}

extern "C" int zs_expert_combine(const void* y, int64_t ldy, int64_t rows, int64_t cols, const int32_t* row_of, const float* weights,
                                 int64_t tokens, int32_t choices, const void* residual, int64_t ldr, void* out, int64_t ldo,
                                 void* stream) {
    static const char* fn = "zs_expert_combine";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    ZS_Q8_TRY(zs::check_routes(fn, tokens, choices, 1));
    ZS_Q8_TRY(check_dim(fn, "rows", rows, 0));
    ZS_Q8_TRY(check_dim(fn, "cols", cols, 1));
    ZS_Q8_TRY(check_bf16(fn, "y", y, ldy, rows, cols));
    ZS_Q8_TRY(zs::check_ints(fn, "row_of", row_of, tokens > 0));
    ZS_Q8_TRY(zs::check_ints(fn, "weights", weights, false));
    if (residual) ZS_Q8_TRY(check_bf16(fn, "residual", residual, ldr, tokens, cols));
    ZS_Q8_TRY(check_bf16(fn, "out", out, ldo, tokens, cols));
    if (tokens == 0) return ZS_OK;
    zs::CombineArgs a{(const uint16_t*)y, (const uint16_t*)residual, ldy, ldr, ldo, rows, cols, tokens, row_of, weights, choices,
                      (int)((cols + 511) / 512), (uint16_t*)out};
    const bool w = wide(y, ldy, 32) && (!residual || wide(residual, ldr, 32)) && wide(out, ldo, 32);
    return cuda_status(fn, zs::launch_kernel(w ? zs::k_expert_combine<true> : zs::k_expert_combine<false>,
                                             dim3(zs::grid_for(tokens * a.chunks, 8)), dim3(256), 0, (cudaStream_t)stream, a));
}

extern "C" int zs_expert_combine_backward(const void* dout, int64_t lddout, const void* y, int64_t ldy, int64_t rows, int64_t cols,
                                          const int32_t* row_of, const float* weights, int64_t tokens, int32_t choices,
                                          const int32_t* starts, const int32_t* counts, int32_t n_experts, const zs_q8* dy,
                                          void* dy_bf16, int64_t lddy, float* dweights, void* stream) {
    static const char* fn = "zs_expert_combine_backward";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::CombineBackArgs a{};
    ZS_Q8_TRY(check_rows(fn, "dy", "dy_bf16", row_of, tokens, choices, starts, counts, n_experts, rows, cols, dy, dy_bf16, lddy, &a.r));
    ZS_Q8_TRY(check_bf16(fn, "dout", dout, lddout, tokens, cols));
    ZS_Q8_TRY(zs::check_ints(fn, "weights", weights, false));
    ZS_Q8_TRY(zs::check_ints(fn, "dweights", dweights, false));
    if (!dy && !dy_bf16 && !dweights) return fail(fn, "dy, dy_bf16 and dweights are all NULL");
    if (dweights) ZS_Q8_TRY(check_bf16(fn, "y", y, ldy, rows, cols));
    if (tokens == 0) return ZS_OK;
    a.dout = (const uint16_t*)dout;
    a.lddout = lddout;
    a.y = (const uint16_t*)y;
    a.ldy = ldy;
    a.weights = weights;
    a.dweights = dweights;
    const bool w = wide(dout, lddout, 32) && (!dweights || wide(y, ldy, 32)) && (!dy_bf16 || wide(dy_bf16, lddy, 32));
    const int group = a.r.chunks < zs::kBackWarps ? a.r.chunks : zs::kBackWarps;
    // a token per CTA, and at least a few CTAs for the rows without one
    const unsigned ctas = tokens < 64 ? 64 : (unsigned)tokens;
    const cudaStream_t st = (cudaStream_t)stream;
    return cuda_status(fn, w ? zs::launch_back<true>(a, ctas, group, st) : zs::launch_back<false>(a, ctas, group, st));
}
