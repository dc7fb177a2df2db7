// C ABI of the e4m3 products, the quantising and the expert routing (declared in
// include/tcl_fp8.h): argument checks, the choice of tile, and the launches.
#include <cuda.h>

#include <algorithm>
#include <cstdint>

#include "fp8_launch.cuh"
#include "tcl_fp8.h"

namespace tcl {
namespace {

constexpr unsigned long long kTimeoutNs = 1000000000ull;   // bound on every in-kernel wait: 1 s

// Counts and widths end here: the kernels round them up to whole tiles, and step past them by up to a
// block's columns, in 32 bits.
constexpr int kMostSize = 0x7ffeffff;

bool sizes(int count0, int count1, int width0, int width1) {
    return count0 >= 0 && count1 >= 0 && width0 >= 1 && width1 >= 1 && std::max(count0, count1) <= kMostSize &&
           std::max(width0, width1) <= kMostSize;
}
bool on(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int elem(int x_type) { return x_type == TCL_X_F32 ? 4 : 2; }
bool known(int x_type) { return x_type == TCL_X_BF16 || x_type == TCL_X_F32; }
long long up(long long x, long long m) { return (x + m - 1) / m * m; }
int groups_of(int k) { return (k + 127) / 128; }

int status_of(cudaError_t err) {
    if (err == cudaSuccess) return TCL_OK;
    cudaGetLastError();
    return err == cudaErrorInvalidValue ? TCL_ERR_DIMS : TCL_ERR_LAUNCH;
}

int device_check() {
    int dev, sms;
    unsigned int* status;
    return device_context(&dev, &sms, &status);
}

// An e4m3 operand as its tensor copies read it.
struct Operand {
    const uint8_t* p;
    long long ld, mat;
    int rows, mats, k;
    bool copy() const { return !on(p, 16) || ld % 16 || (mats > 1 && mat % 16); }
    size_t bytes() const { return copy() ? static_cast<size_t>(up(static_cast<long long>(mats) * rows * up(k, 16), 256)) : 0; }
};

// Copies an operand that is off the tensor copies' grid into `to`.
int lay_out(Operand& o, uint8_t* to, cudaStream_t stream) {
    if (!o.copy()) return TCL_OK;
    const long long ld = up(o.k, 16);
    const cudaError_t err = launch_copy_bytes(o.p, o.ld, o.mat, to, ld, o.mats, o.rows, o.k, stream);
    if (err != cudaSuccess) return status_of(err);
    o.p = to;
    o.ld = ld;
    o.mat = ld * o.rows;
    return TCL_OK;
}

// The tile for products of `tokens` rows with N columns, for `experts` experts. Few rows go to
// the MMA's N side, many to its M side. Measured in CUDA graphs on a GB300, microseconds:
//   dense, N = K = 4096     M =  8    64   128   256   512  1024  2048
//     128 × 16                 7.0  12.1  14.0  24.3  42.6
//     128 × 32                 8.0  10.9  15.1  16.5  28.4
//     128 × 128               15.6  15.3  15.2  15.5  16.0  27.5  49.7   (10.4 and 14.0 at M = 128
//                                                       and 256 since clusters share their k-blocks)
//     256 × 256, two SMs                        18.8  19.2  19.4  33.2
//   64 experts, N = 4096, K = 2048: rows each (on average)
//                               1/8     2     8    16    32    64   128   256   512
//     128 × 16                 11.9  51.6  72.3  85.4   106   173   313
//     128 × 32                 15.6  52.0  71.8  81.6  92.1   123   210
//     128 × 128                30.1  57.0  82.4  90.3  96.4   113   143   216   386
//     256 × 256, two SMs                               122   123   140   184   275
// (128 × 64 tiles were within 5 % of the best of these everywhere.) So 128 × 128 tiles from some
// dozen rows until they need a second wave of the GPU, then 256 × 256 (not for experts of about
// a hundred rows, which leave most of such a tile empty: at 96 rows 132 us against 127).
Fp8Tile choose_tile(long long tokens, int experts, int N, int sms) {
    const long long each = (tokens + experts - 1) / experts;
    const long long ones = (each + 127) / 128 * ((N + 127) / 128) * experts;
    if (each <= (experts == 1 ? 16 : 4)) return Fp8Tile::FEW16;
    if (each <= (experts == 1 ? 64 : 40)) return Fp8Tile::FEW32;
    if (each > 112 && N > 128 && ones > sms) return Fp8Tile::PAIR;
    return Fp8Tile::ONE;
}

int product(Operand a, Fp8Side sa, Operand b, Fp8Side sb, Fp8Tile tile, Fp8Params p, long long units, int sms,
            cudaStream_t stream) {
    const auto lock = library_lock();   // (to the launch below)
    if (const size_t need = a.bytes() + b.bytes()) {
        void* scratch;
        int st = stream_scratch(stream, need, &scratch);
        if (st) return st;
        uint8_t* at = static_cast<uint8_t*>(scratch);
        const size_t first = a.bytes();
        if ((st = lay_out(a, at, stream)) || (st = lay_out(b, at + first, stream))) return st;
    }
    const Fp8TileInfo t = fp8_tile_info(tile);
    // P is the side in the tensor-memory lanes: the tokens, or few tokens' weights
    const Operand& op = t.swap ? b : a;
    const Operand& oq = t.swap ? a : b;
    Fp8Launch l;
    l.tile = tile;
    int st;
    if ((st = tensor_map_bytes(op.p, op.k, op.rows, op.mats, op.ld, op.mats > 1 ? op.mat : up(op.ld * op.rows, 16),
                               t.box_p, &l.tmP)) ||
        (st = tensor_map_bytes(oq.p, oq.k, oq.rows, oq.mats, oq.ld, oq.mats > 1 ? oq.mat : up(oq.ld * oq.rows, 16),
                               t.box_q, &l.tmQ)))
        return st;
    if (p.vec && !t.swap) {
        const int es = p.out_bf16 ? 2 : 4;
        const long long rows = p.wgrad ? p.wrows : p.rows, cols = p.wgrad ? p.qrows : p.wrows;
        if ((st = tensor_map_result(p.C, p.out_bf16, cols, rows, p.wgrad ? p.experts : 1, p.ldc * es,
                                    p.wgrad && p.experts > 1 ? p.c_expert * es : p.ldc * es * rows, &l.tmC)))
            return st;
    }
    p.P = t.swap ? sb : sa;
    p.Q = t.swap ? sa : sb;
    p.timeout_ns = kTimeoutNs;
    int ctas = t.ctas;
    const int places = sms * t.per_sm;
    p.split = 1;
    if (t.ctas == 1) {
        // share tiles while every CTA has a place and enough to do: two k-blocks of a narrow tile,
        // eight of a 128 × 128 one, whose sums take longer to exchange (1000 × 776 × 1030 with
        // four or five each 10.8 us, whole 9.2; 128 × 4096 × 4096 with eight each 10.5, whole 15.2)
        const int least = t.swap ? 2 : 8, kbs = p.wgrad ? p.rows / 128 / p.experts : p.num_kb;
        while (p.split < 8 && units * p.split * 2 <= places && kbs >= p.split * 2 * least) p.split *= 2;
        ctas = p.split;
    }
    l.p = p;
    l.grid = static_cast<int>(std::max(1ll, std::min<long long>(places / ctas, units))) * ctas;
    l.stream = stream;
    return status_of(launch_fp8_gemm(l));
}

// Rows of tokens times the weights of one matrix (offsets NULL) or of each row's expert.
int rows_product(int rows, int experts, int N, int K, const void* A, int lda, const float* SA, long long sa_row,
                 long long sa_group, const void* B, int ldb, long long b_expert, const float* SB, int sb_kind,
                 long long sb_expert, long long sb_row, long long sb_group, const int32_t* offsets, void* C, int ldc,
                 int out, cudaStream_t stream) {
    if (!sizes(rows, 0, N, K) || experts < 1) return TCL_ERR_DIMS;
    if (experts > TCL_MAX_EXPERTS) return TCL_ERR_CONFIG;
    if (out != TCL_OUT_F32 && out != TCL_OUT_BF16) return TCL_ERR_CONFIG;
    if (sb_kind != TCL_SCALE_ROWS && sb_kind != TCL_SCALE_BLOCKS) return TCL_ERR_CONFIG;
    if (!B || !SB || (rows && (!A || !SA || !C))) return TCL_ERR_NULL;
    if (lda < K || ldb < K || ldc < N) return TCL_ERR_LD;
    if (experts > 1 && b_expert < static_cast<long long>(N - 1) * ldb + K) return TCL_ERR_LD;
    const int es = out == TCL_OUT_BF16 ? 2 : 4;
    if (!on(SA, 4) || !on(SB, 4) || !on(C, es) || !on(offsets, 4)) return TCL_ERR_ALIGN;
    int dev, sms;
    unsigned int* status;
    int st = device_context(&dev, &sms, &status);
    if (st) return st;
    if (rows == 0) return TCL_OK;
    const Fp8Tile tile = choose_tile(rows, experts, N, sms);
    const Fp8TileInfo t = fp8_tile_info(tile);
    const int tt = t.swap ? t.bq : t.bp, tw = t.swap ? t.bp : t.bq;
    Fp8Params p = {};
    p.offsets = offsets;
    p.experts = experts;
    p.rows = rows;
    p.wrows = N;
    p.num_kb = groups_of(K);
    p.C = C;
    p.ldc = ldc;
    p.out_bf16 = out == TCL_OUT_BF16;
    p.vec = on(C, 16) && static_cast<long long>(ldc) * es % 16 == 0;
    p.status = status;
    // (every expert may end inside a tile, and so may the rows behind the last)
    const long long units = (offsets ? static_cast<long long>(rows) / tt + 1 + std::min(experts, rows)
                                     : (static_cast<long long>(rows) + tt - 1) / tt) *
                            ((N + tw - 1) / tw);
    if (units > 0x3fffffffll) return TCL_ERR_DIMS;
    return product({static_cast<const uint8_t*>(A), lda, 0, rows, 1, K}, {SA, sa_row, sa_group, 0, 0},
                   {static_cast<const uint8_t*>(B), ldb, b_expert, N, experts, K},
                   {SB, sb_row, sb_group, experts > 1 ? sb_expert : 0, sb_kind}, tile, p, units, sms, stream);
}

}  // namespace
}  // namespace tcl

using namespace tcl;

extern "C" {

int tcl_quantize_fp8_rows(int x_type, int rows, int cols, const void* X, int ldx, const int32_t* position, int top,
                          const int32_t* source, int out_rows, void* Q, int ldq, float* scale, long long s_row,
                          long long s_group, cudaStream_t stream) {
    if (!known(x_type)) return TCL_ERR_CONFIG;
    const int made = position ? out_rows : rows;
    if (!sizes(rows, made, cols, 1) || (position && top < 1)) return TCL_ERR_DIMS;
    if ((rows && !X) || (made && (!Q || !scale)) || (position && made && !source)) return TCL_ERR_NULL;
    if (ldx < cols || ldq < cols) return TCL_ERR_LD;
    if (!on(X, elem(x_type)) || !on(scale, 4) || !on(position, 4) || !on(source, 4)) return TCL_ERR_ALIGN;
    if (int st = device_check()) return st;
    if (made == 0) return TCL_OK;
    return status_of(launch_quant_rows({X, ldx, x_type == TCL_X_F32, rows, cols, position, top, source, out_rows,
                                        static_cast<uint8_t*>(Q), ldq, scale, s_row, s_group},
                                       stream));
}

int tcl_quantize_fp8_columns(int x_type, int rows, int cols, const void* X, int ldx, const int32_t* source, int top,
                             int out_rows, void* Q, int ldq, float* scale, long long s_row, long long s_group,
                             cudaStream_t stream) {
    if (!known(x_type)) return TCL_ERR_CONFIG;
    const int made = source ? out_rows : rows;
    if (!sizes(rows, made, cols, 1) || (source && top < 1)) return TCL_ERR_DIMS;
    if ((rows && !X) || (made && (!Q || !scale))) return TCL_ERR_NULL;
    if (ldx < cols || ldq < made) return TCL_ERR_LD;
    if (!on(X, elem(x_type)) || !on(scale, 4) || !on(source, 4)) return TCL_ERR_ALIGN;
    if (int st = device_check()) return st;
    if (made == 0) return TCL_OK;
    return status_of(launch_quant_tiles(QuantTile::COLUMNS,
                                        {X, ldx, 0, x_type == TCL_X_F32, 1, made, cols, rows, source, top,
                                         static_cast<uint8_t*>(Q), ldq, 0, scale, 0, s_row, s_group},
                                        stream));
}

int tcl_quantize_fp8_blocks(int x_type, int batch, int rows, int cols, const void* X, int ldx, long long x_batch,
                            int transpose, void* Q, int ldq, long long q_batch, float* scale, cudaStream_t stream) {
    if (!known(x_type) || (transpose != 0 && transpose != 1)) return TCL_ERR_CONFIG;
    if (!sizes(batch, rows, cols, 1)) return TCL_ERR_DIMS;
    const bool any = batch > 0 && rows > 0;
    if (any && (!X || !Q || !scale)) return TCL_ERR_NULL;
    const int qrows = transpose ? cols : rows, qcols = transpose ? rows : cols;
    if (ldx < cols || ldq < qcols) return TCL_ERR_LD;
    if (batch > 1 && any && (x_batch < 0 || q_batch < static_cast<long long>(qrows - 1) * ldq + qcols)) return TCL_ERR_LD;
    if (!on(X, elem(x_type)) || !on(scale, 4)) return TCL_ERR_ALIGN;
    if (int st = device_check()) return st;
    if (!any) return TCL_OK;
    const long long groups = groups_of(qcols);   // (the scales lie one matrix after another)
    return status_of(launch_quant_tiles(transpose ? QuantTile::BLOCKS_T : QuantTile::BLOCKS,
                                        {X, ldx, x_batch, x_type == TCL_X_F32, batch, rows, cols, rows, nullptr, 1,
                                         static_cast<uint8_t*>(Q), ldq, q_batch, scale, groups_of(qrows) * groups, groups, 1},
                                        stream));
}

int gemm_fp8(int M, int N, int K, const void* A, int lda, const float* SA, long long sa_row, long long sa_group,
             const void* B, int ldb, const float* SB, int sb_kind, long long sb_row, long long sb_group, void* C, int ldc,
             int out, cudaStream_t stream) {
    return rows_product(M, 1, N, K, A, lda, SA, sa_row, sa_group, B, ldb, 0, SB, sb_kind, 0, sb_row, sb_group, nullptr, C,
                        ldc, out, stream);
}

int gemm_fp8_experts(int rows, int experts, int N, int K, const void* A, int lda, const float* SA, long long sa_row,
                     long long sa_group, const void* B, int ldb, long long b_expert, const float* SB, int sb_kind,
                     long long sb_expert, long long sb_row, long long sb_group, const int32_t* offsets, void* C, int ldc,
                     int out, cudaStream_t stream) {
    if (!offsets) return TCL_ERR_NULL;
    return rows_product(rows, experts, N, K, A, lda, SA, sa_row, sa_group, B, ldb, b_expert, SB, sb_kind, sb_expert,
                        sb_row, sb_group, offsets, C, ldc, out, stream);
}

int gemm_fp8_experts_wgrad(int rows, int experts, int N, int K, const void* A, int lda, const float* SA, long long sa_row,
                           long long sa_group, const void* B, int ldb, const float* SB, long long sb_row,
                           long long sb_group, const int32_t* offsets, void* C, int ldc, long long c_expert, int out,
                           cudaStream_t stream) {
    if (!sizes(rows, 0, N, K) || experts < 1) return TCL_ERR_DIMS;
    if (experts > TCL_MAX_EXPERTS) return TCL_ERR_CONFIG;
    if (out != TCL_OUT_F32 && out != TCL_OUT_BF16) return TCL_ERR_CONFIG;
    if (!offsets || !C || (rows && (!A || !SA || !B || !SB))) return TCL_ERR_NULL;
    if (lda < rows || ldb < rows || ldc < K) return TCL_ERR_LD;
    if (experts > 1 && c_expert < static_cast<long long>(N - 1) * ldc + K) return TCL_ERR_LD;
    const int es = out == TCL_OUT_BF16 ? 2 : 4;
    if (!on(SA, 4) || !on(SB, 4) || !on(C, es) || !on(offsets, 4)) return TCL_ERR_ALIGN;
    int dev, sms;
    unsigned int* status;
    int st = device_context(&dev, &sms, &status);
    if (st) return st;
    if (rows == 0) {   // no expert has rows: all zeros
        for (int e = 0; e < experts; ++e)
            if (cudaMemset2DAsync(static_cast<char*>(C) + e * c_expert * es, static_cast<size_t>(ldc) * es, 0,
                                  static_cast<size_t>(K) * es, N, stream) != cudaSuccess)
                return status_of(cudaErrorUnknown);
        return TCL_OK;
    }
    // (as above: 256 × 256 tiles once 128 × 128 ones need a second wave)
    const long long ones = static_cast<long long>(experts) * ((N + 127) / 128) * ((K + 127) / 128);
    const Fp8Tile tile = N > 128 && K > 128 && ones > sms ? Fp8Tile::PAIR : Fp8Tile::ONE;
    const Fp8TileInfo t = fp8_tile_info(tile);
    Fp8Params p = {};
    p.offsets = offsets;
    p.experts = experts;
    p.rows = rows;
    p.wrows = N;
    p.qrows = K;
    p.wgrad = 1;
    p.C = C;
    p.ldc = ldc;
    p.c_expert = c_expert;
    p.out_bf16 = out == TCL_OUT_BF16;
    p.vec = on(C, 16) && static_cast<long long>(ldc) * es % 16 == 0 && (experts == 1 || c_expert * es % 16 == 0);
    p.status = status;
    const long long units = static_cast<long long>(experts) * ((N + t.bp - 1) / t.bp) * ((K + t.bq - 1) / t.bq);
    if (units > 0x3fffffffll) return TCL_ERR_DIMS;
    return product({static_cast<const uint8_t*>(A), lda, 0, N, 1, rows}, {SA, sa_row, sa_group, 0, 0},
                   {static_cast<const uint8_t*>(B), ldb, 0, K, 1, rows}, {SB, sb_row, sb_group, 0, 0}, tile, p, units, sms,
                   stream);
}

int tcl_sort_by_expert(int tokens, int top, const void* ids, int id_bytes, int experts, int align, int rows,
                       int32_t* offsets, int32_t* position, int32_t* source, cudaStream_t stream) {
    if (id_bytes != 4 && id_bytes != 8) return TCL_ERR_CONFIG;
    if (experts > TCL_MAX_EXPERTS || align < 1 || align > 128) return TCL_ERR_CONFIG;
    if (!sizes(tokens, std::max(rows, 0), top, experts)) return TCL_ERR_DIMS;
    const long long slots = static_cast<long long>(tokens) * top;
    const long long need = (slots + std::min<long long>(experts, slots) * (align - 1)) / align * align;
    if (need > kMostSize || rows < need) return TCL_ERR_DIMS;
    if (!offsets || (slots && (!ids || !position)) || (rows && !source)) return TCL_ERR_NULL;
    if (!on(ids, id_bytes) || !on(offsets, 4) || !on(position, 4) || !on(source, 4)) return TCL_ERR_ALIGN;
    if (int st = device_check()) return st;
    return status_of(launch_sort(slots, ids, id_bytes, experts, align, rows, offsets, position, source, stream));
}

int tcl_gather_rows(int x_type, int tokens, int top, int rows, int cols, const void* X, int ldx, const int32_t* position,
                    const int32_t* source, void* Y, int ldy, cudaStream_t stream) {
    if (!known(x_type)) return TCL_ERR_CONFIG;
    if (!sizes(tokens, rows, top, cols)) return TCL_ERR_DIMS;
    if ((tokens && (!X || !position)) || (rows && (!Y || !source))) return TCL_ERR_NULL;
    if (ldx < cols || ldy < cols) return TCL_ERR_LD;
    if (!on(X, elem(x_type)) || !on(Y, elem(x_type)) || !on(position, 4) || !on(source, 4)) return TCL_ERR_ALIGN;
    if (int st = device_check()) return st;
    if (rows == 0) return TCL_OK;
    RouteRows a = {};
    a.f32 = x_type == TCL_X_F32;
    a.tokens = tokens, a.top = top, a.rows = rows, a.cols = cols;
    a.x = X, a.ldx = ldx;
    a.position = position, a.source = source;
    a.out = Y, a.ldo = ldy;
    return status_of(launch_gather(a, stream));
}

int tcl_combine(int x_type, int tokens, int top, int rows, int cols, const void* Y, int ldy, const float* weights,
                const int32_t* position, void* out, int ldo, cudaStream_t stream) {
    if (!known(x_type)) return TCL_ERR_CONFIG;
    if (!sizes(tokens, rows, top, cols)) return TCL_ERR_DIMS;
    if ((tokens && (!out || !position)) || (rows && !Y)) return TCL_ERR_NULL;
    if (ldy < cols || ldo < cols) return TCL_ERR_LD;
    if (!on(Y, elem(x_type)) || !on(out, elem(x_type)) || !on(weights, 4) || !on(position, 4)) return TCL_ERR_ALIGN;
    if (int st = device_check()) return st;
    RouteRows a = {};
    a.f32 = x_type == TCL_X_F32;
    a.tokens = tokens, a.top = top, a.rows = rows, a.cols = cols;
    a.x = Y, a.ldx = ldy;
    a.weights = weights;
    a.position = position;
    a.out = out, a.ldo = ldo;
    return status_of(launch_combine(a, stream));
}

int tcl_combine_grad(int x_type, int tokens, int top, int rows, int cols, const void* G, int ldg, const void* Y, int ldy,
                     const float* weights, const int32_t* position, const int32_t* source, void* DY, int lddy, float* DW,
                     cudaStream_t stream) {
    if (!known(x_type)) return TCL_ERR_CONFIG;
    if (!sizes(tokens, rows, top, cols)) return TCL_ERR_DIMS;
    if ((tokens && (!G || !position)) || (DY && rows && !source) || (DW && rows && !Y)) return TCL_ERR_NULL;
    if (ldg < cols || (DW && ldy < cols) || (DY && lddy < cols)) return TCL_ERR_LD;
    if (!on(G, elem(x_type)) || !on(Y, elem(x_type)) || !on(DY, elem(x_type)) || !on(DW, 4) || !on(weights, 4) ||
        !on(position, 4) || !on(source, 4))
        return TCL_ERR_ALIGN;
    if (int st = device_check()) return st;
    if (!DY && !DW) return TCL_OK;
    RouteRows a = {};
    a.f32 = x_type == TCL_X_F32;
    a.tokens = tokens, a.top = top, a.rows = rows, a.cols = cols;
    a.x = G, a.ldx = ldg;
    a.y = Y, a.ldy = ldy;
    a.weights = weights;
    a.position = position, a.source = source;
    a.out = DY, a.ldo = lddy;
    a.dw = DW;
    return status_of(launch_combine_grad(a, stream));
}

}  // extern "C"
