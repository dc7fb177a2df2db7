// Internal launch interface of the e4m3 products and of the kernels around them:
// what api_fp8.cu needs of the translation units that hold the kernels, and of api.cu.
#pragma once

#include <cuda_runtime.h>

#include <mutex>

#include "fp8_gemm.cuh"

namespace tcl {

// ---- services of api.cu
int device_context(int* dev, int* sms, unsigned int** status);
// The lock of the library's state. A call holds it from its scratch to the last launch that uses it, so
// that another thread's call on the stream cannot come in between; what follows is called under it.
std::unique_lock<std::mutex> library_lock();
// `need` bytes of the library scratch that belongs to `stream` (grown on demand; TCL_ERR_CAPTURE inside a capture).
int stream_scratch(cudaStream_t stream, size_t need, void** out);
// A 3-D map of bytes (K contiguous, rows, matrices), 128-byte swizzle, boxes of 128 bytes × box_rows; not cached.
int tensor_map_bytes(const void* ptr, uint64_t k, uint64_t rows, uint64_t mats, uint64_t row_stride, uint64_t mat_stride,
                     uint32_t box_rows, CUtensorMap* out);
// The same for a product's result (fp32 or bf16), boxes of 128 bytes × 32 rows.
int tensor_map_result(const void* ptr, int bf16, uint64_t cols, uint64_t rows, uint64_t mats, uint64_t row_stride,
                      uint64_t mat_stride, CUtensorMap* out);

// ---- fp8 products (k_fp8_gemm.cu)
enum class Fp8Tile : int {
    FEW16,    // 128 weight rows × 16 token rows
    FEW32,    // ... × 32
    ONE,      // 128 × 128 on one SM
    PAIR,     // 256 × 256 on a pair of SMs
};
struct Fp8Launch {
    Fp8Tile tile;
    CUtensorMap tmP, tmQ, tmC;
    Fp8Params p;
    int grid;
    cudaStream_t stream;
};
struct Fp8TileInfo {
    int bp, bq, ctas, box_p, box_q, swap, per_sm;
};
Fp8TileInfo fp8_tile_info(Fp8Tile t);
cudaError_t launch_fp8_gemm(const Fp8Launch& a);

// Launches with programmatic stream serialisation: the kernel's set-up may overlap the end of the
// kernel before it in the stream (it waits for that kernel before it touches global memory).
template <class... KArgs, class... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// ---- quantising (k_quantize.cu)
struct QuantRows {
    const void* x;
    long long ldx;
    int f32;                 // X is fp32 (else bf16)
    int rows, cols;
    const int* position;     // tokens' rows in the sorted layout (NULL: row i to row i)
    int top;
    const int* source;
    int out_rows;
    uint8_t* q;
    long long ldq;
    float* scale;
    long long s_row, s_group;
};
cudaError_t launch_quant_rows(const QuantRows& a, cudaStream_t stream);

enum class QuantTile : int { COLUMNS, BLOCKS, BLOCKS_T };
struct QuantTiles {
    const void* x;
    long long ldx, x_batch;
    int f32;
    int batch, rows, cols;   // rows of the layout (length of source where there is one)
    int x_rows;              // rows of X
    const int* source;
    int top;
    uint8_t* q;
    long long ldq, q_batch;
    float* scale;
    long long s_batch, s_row, s_group;
    long long room;          // of Q's rows from q on (set by the launch)
};
cudaError_t launch_quant_tiles(QuantTile kind, const QuantTiles& a, cudaStream_t stream);

// dst[b][r][c] = src[b][r][c], bytes, any alignment of src.
cudaError_t launch_copy_bytes(const uint8_t* src, long long ld, long long batch_stride, uint8_t* dst, long long ld_dst,
                              int batch, int rows, int cols, cudaStream_t stream);

// ---- routing (k_route.cu)
constexpr int kSortChunk = 4096;   // most slots of one block
cudaError_t launch_sort(long long slots, const void* ids, int id_bytes, int experts, int align, int rows, int* offsets,
                        int* position, int* source, cudaStream_t stream);

struct RouteRows {
    int f32;
    int tokens, top, rows, cols;
    const void* x;           // tokens' rows (combine: the sorted rows)
    long long ldx;
    const void* y;           // combine_grad: the sorted rows
    long long ldy;
    const float* weights;
    const int* position;
    const int* source;
    void* out;
    long long ldo;
    float* dw;
};
cudaError_t launch_gather(const RouteRows& a, cudaStream_t stream);
cudaError_t launch_combine(const RouteRows& a, cudaStream_t stream);
cudaError_t launch_combine_grad(const RouteRows& a, cudaStream_t stream);

}  // namespace tcl
