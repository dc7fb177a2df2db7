// Internal launch interface of the dense bf16 products with fused ends and of the passes around
// them: what api_dense.cu needs of the translation units that hold the kernels, and of api.cu.
#pragma once

#include <cuda_runtime.h>

#include "dense_few.cuh"
#include "fp8_launch.cuh"

namespace tcl {

// ---- services of api.cu (under the library's lock)
// A 2-D map of a stored bf16 matrix (cols contiguous), 128-byte swizzle, boxes of 64 columns × box_rows.
int tensor_map_bf16(const void* ptr, uint64_t cols, uint64_t rows, uint64_t row_bytes, uint32_t box_rows, CUtensorMap* out);
// The same matrix as chunks of 64 columns: a 3-D map (64 columns, rows, chunks), boxes of 64 × box_rows × box_chunks.
int tensor_map_bf16_chunks(const void* ptr, uint64_t chunks, uint64_t rows, uint64_t row_bytes, uint32_t box_rows,
                           uint32_t box_chunks, CUtensorMap* out);

// ---- products (k_dense.cu, k_dense_few.cu)
struct DenseLaunch {
    DenseEnd end;
    int bn;              // 256 or 128: columns of a tile
    DenseMaps maps;
    DenseParams p;
    int pairs;
    cudaStream_t stream;
};
cudaError_t launch_dense_pair(const DenseLaunch& a);

struct DenseFewLaunch {
    DenseEnd end;
    int bq;              // 16, 32, 64 or 128
    CUtensorMap w[2], x;
    DenseFewParams p;
    int grid;
    cudaStream_t stream;
};
// Clusters of `split` (1, 2, 4 or 8) of its CTAs that the GPU holds at once: fewer than its SMs would do for, since
// a cluster stays within a group of SMs.
int dense_few_clusters(int split, int sms);
cudaError_t launch_dense_few(const DenseFewLaunch& a);

// ---- passes (k_dense_rows.cu)
struct DenseCopy {       // rows × cols of bf16 to rows of whole 16-byte pieces
    const __nv_bfloat16* from;
    long long ld;
    int rows, cols;
    __nv_bfloat16* to;
    long long ld_to;
};
constexpr int kDenseCopies = 6;
struct DenseCopies {
    DenseCopy job[kDenseCopies];
    int n;
};
cudaError_t launch_dense_copies(const DenseCopies& a, cudaStream_t stream);

struct DenseJoin {       // the sums of K ranges, added in their order
    const float* parts;
    long long ld, part;  // elements between rows, between ranges
    int splits, rows, cols, f32;
    const float* factor;
    const float* plus;
    long long ld_plus;
    void* out;
    long long ld_out;
};
cudaError_t launch_dense_join(const DenseJoin& a, cudaStream_t stream);

struct EntropyRows {
    const float2* parts;   // [chunk][row]
    int chunks, chunk, rows, vocab;   // chunk: columns of e of one sum (in training)
    const float* target_logit;
    const void* targets;
    int wide_targets;
    float *loss, *lse;
    const __nv_bfloat16 *x, *w;   // their rows, on 16-byte pieces
    long long ld_x, ld_w;
    int hidden;
    // in training:
    const float* grad;     // NULL: no gradients
    __nv_bfloat16* e;      // exponentials
    long long ld_e;
    float* factor;
    __nv_bfloat16* scaled;
    long long ld_scaled;
};
cudaError_t launch_entropy_rows(const EntropyRows& a, cudaStream_t stream);

}  // namespace tcl
