// Internal launch interface of the gradients' norm and clipping.
#pragma once

#include <cuda_runtime.h>

namespace tcl {

constexpr int kClipTensors = 256;          // of one launch (they travel in its parameters)
constexpr int kClipBlocks = 152 * 8;

struct ClipTensor {
    const void* from;
    void* to;
    long long n, before;   // elements; pieces of the tensors before it
};
struct ClipTensors {
    ClipTensor t[kClipTensors];
    int n, f32;
    int piece;                         // elements that a block takes at a time
    long long pieces;
};
// Sums of squares: parts[block], one for each of clip_blocks(a.pieces) blocks.
int clip_blocks(long long pieces);
cudaError_t launch_square_sums(const ClipTensors& a, double* parts, cudaStream_t stream);
// norm = sqrt of the sum of n parts.
cudaError_t launch_norm(const double* parts, int n, float* norm, cudaStream_t stream);
// to = from · (bound / norm if norm > bound, else 1); norm from n parts, written if it is given.
cudaError_t launch_clip(const ClipTensors& a, const double* parts, int n, float bound, float* norm, cudaStream_t stream);

}  // namespace tcl
