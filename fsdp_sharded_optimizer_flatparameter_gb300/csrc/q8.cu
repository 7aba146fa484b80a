// The 8-bit format's own calls: encode (as it is, transposed, or both), decode, and the transpose of a
// kept matrix.  All move bytes: encode reads 2 bytes per value and writes 1 or 2, the transpose reads 1
// and writes 1, decode reads 1 and writes 2.
#include "q8_tile.cuh"

namespace zs {

namespace {

struct DecodeArgs {
    Q8 q;
    uint16_t* y;
    int64_t ldy, rows, cols, chunks;     // chunks of 16 columns per row
    int wide;
};

__global__ void __launch_bounds__(256) k_q8_decode(const __grid_constant__ DecodeArgs a) {
    dependent_launch_prologue();
    const int64_t i = gtid();
    const int64_t r = i / a.chunks, c = (i - r * a.chunks) * 16;
    if (r >= a.rows) return;
    const int n = a.cols - c < 16 ? (int)(a.cols - c) : 16;
    const uint4 w = load_codes(a.q.codes + r * a.q.ld + c, n);
    const float s = q8_scale(a.q.scales[r * a.q.lds + (c >> 7)]);
    float f[16];
    q8_unpack4(w.x, s, f);
    q8_unpack4(w.y, s, f + 4);
    q8_unpack4(w.z, s, f + 8);
    q8_unpack4(w.w, s, f + 12);
    uint16_t* y = a.y + r * a.ldy + c;
    if (a.wide && n == 16) {
        reinterpret_cast<uint4*>(y)[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                    pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        reinterpret_cast<uint4*>(y)[1] = make_uint4(pack_bf16x2(f[8], f[9]), pack_bf16x2(f[10], f[11]),
                                                    pack_bf16x2(f[12], f[13]), pack_bf16x2(f[14], f[15]));
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < n) y[j] = f32_to_bf16(f[j]);
    }
}

}  // namespace

}  // namespace zs

using namespace zs::q8_host;

extern "C" int zs_set_q8_wait_limit(int64_t limit_cycles) {
    zs::clear_error();
    if (limit_cycles < 0 || limit_cycles > (int64_t(1) << 32)) return fail("zs_set_q8_wait_limit", "limit_cycles out of range");
    zs::wait_limit().store((long long)limit_cycles, std::memory_order_relaxed);
    return ZS_OK;
}

extern "C" int zs_q8_encode(const void* x, int64_t ldx, int64_t rows, int64_t cols, const zs_q8* q, const zs_q8* q_t,
                            void* stream) {
    static const char* fn = "zs_q8_encode";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::TileArgs a{};
    ZS_Q8_TRY(check_dim(fn, "rows", rows, 0));
    ZS_Q8_TRY(check_dim(fn, "cols", cols, 1));
    ZS_Q8_TRY(check_bf16(fn, "x", x, ldx, rows, cols));
    ZS_Q8_TRY(check_q8(fn, "q", q, rows, cols, true, &a.rows_out[0]));
    ZS_Q8_TRY(check_q8(fn, "q_t", q_t, cols, rows, true, &a.cols_out[0]));
    if (!q && !q_t) return fail(fn, "q and q_t are both NULL");
    if (rows == 0) return ZS_OK;
    a.x = (const uint16_t*)x;
    a.ldx = ldx;
    a.rows = rows;
    a.cols = cols;
    const cudaStream_t st = (cudaStream_t)stream;
    return cuda_status(fn, wide(x, ldx) ? zs::launch_tiles<zs::kTileEncode, true>(a, st) : zs::launch_tiles<zs::kTileEncode, false>(a, st));
}

extern "C" int zs_q8_transpose(const zs_q8* q, int64_t rows, int64_t cols, const zs_q8* q_t, void* stream) {
    static const char* fn = "zs_q8_transpose";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::TileArgs a{};
    ZS_Q8_TRY(check_dim(fn, "rows", rows, 0));
    ZS_Q8_TRY(check_dim(fn, "cols", cols, 1));
    ZS_Q8_TRY(check_q8(fn, "q", q, rows, cols, false, &a.a));
    ZS_Q8_TRY(check_q8(fn, "q_t", q_t, cols, rows, false, &a.cols_out[0]));
    if (rows == 0) return ZS_OK;
    a.rows = rows;
    a.cols = cols;
    return cuda_status(fn, zs::launch_tiles<zs::kTileTurn, true>(a, (cudaStream_t)stream));
}

extern "C" int zs_q8_decode(const zs_q8* q, int64_t rows, int64_t cols, void* y, int64_t ldy, void* stream) {
    static const char* fn = "zs_q8_decode";
    zs::TraceRange trace_(fn);
    zs::clear_error();
    zs::DecodeArgs a{};
    ZS_Q8_TRY(check_dim(fn, "rows", rows, 0));
    ZS_Q8_TRY(check_dim(fn, "cols", cols, 1));
    ZS_Q8_TRY(check_q8(fn, "q", q, rows, cols, false, &a.q));
    ZS_Q8_TRY(check_bf16(fn, "y", y, ldy, rows, cols));
    if (rows == 0) return ZS_OK;
    a.y = (uint16_t*)y;
    a.ldy = ldy;
    a.rows = rows;
    a.cols = cols;
    a.chunks = (cols + 15) / 16;
    a.wide = wide(y, ldy);
    const int64_t blocks = (rows * a.chunks + 255) / 256;
    if (blocks > 0x7fffffffLL) return fail(fn, "matrix too large for one launch");
    return cuda_status(fn, zs::launch_kernel(zs::k_q8_decode, dim3((unsigned)blocks), dim3(256), 0,
                                             (cudaStream_t)stream, a));
}
