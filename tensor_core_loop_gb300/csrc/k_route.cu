// Tokens sorted by expert and back: the order, the rows laid out in it, the weighted sum of
// the experts' rows, and its gradients.
//
// The order is a counting sort by expert that keeps the slots' order. A block takes up to 4,096
// slots, each of its 32 warps 128 consecutive ones. Counts of a warp, then of the warps
// before it, then of the blocks before it give every slot its row without an atomic whose
// order could show in the result (the shared-memory atomics below only add counts). One
// block needs one launch. More need two before it: each block's counts, and for every expert
// their running sums over the blocks, so that a block reads its own share alone (adding up all
// blocks' counts in every block took 2.3 ms for 8.4 million slots). What passes between the
// launches lies in the outputs that the last one fills: the counts in `source`, a block's sums
// in its own slots of `position`. A sort keeps no memory of its own, so sorts on any streams, from
// any threads and in graphs that replay beside them stay apart. It reads 4 or 8 bytes
// and writes 4 for each slot and writes 4 for each row: launches, not bytes, take the time
// (131,072 slots, 64 experts: 13 us; 8.4 million, 256 experts: 225).
//
// The row kernels are bound by memory: a thread handles eight columns, and a token's row
// (gather, gradient of combine) is read once for all of its slots. 8191 tokens × 6 slots of
// 4096 bf16: combine 81 us, 5.8 TB/s, its gradients 154 us, 6.1 TB/s; 16384 × 8 gathered
// 206 us, 6.2 TB/s. fp32: 132 us, 7.1 TB/s; 300 us, 6.3; gathered 565 us, 4.5 TB/s, for a reason that
// has not been looked for. The gradients' kernel of bf16 rows at any address spills 68 bytes.
#include <algorithm>

#include "fp8_launch.cuh"
#include "rows8.cuh"

namespace tcl {
namespace {

constexpr int kSortThreads = 1024, kSortWarps = 32, kPerLane = kSortChunk / kSortThreads;

template <typename ID>
__device__ __forceinline__ int expert_of(const ID* ids, long long i, long long slots, int experts) {
    if (i >= slots) return -1;
    const ID v = ids[i];
    return v >= 0 && v < experts ? static_cast<int>(v) : -1;
}

// The slots of block b of `blocks`, dealt out evenly: more than 2,048 of them where there are two
// blocks or more, so that a block's slots of `position` hold two numbers for every expert.
__device__ __forceinline__ long long first_slot(long long slots, int b, int blocks) { return slots * b / blocks; }
static_assert(2 * kMaxExperts <= kSortChunk / 2, "a block's running sums fit its slots");

// counts[block][expert]
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const ID* ids, long long slots, int experts,
                                                                  int* counts) {
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < experts; e += kSortThreads) hist[e] = 0;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    __syncthreads();
    const long long base = first_slot(slots, blockIdx.x, gridDim.x), end = first_slot(slots, blockIdx.x + 1, gridDim.x);
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        const int e = expert_of(ids, base + k * kSortThreads + threadIdx.x, end, experts);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kSortThreads)
        counts[static_cast<long long>(blockIdx.x) * experts + e] = hist[e];
}

// 32 experts to a block, a lane each; a warp takes a run of the sort's blocks. Into each block's
// slots of `position`: [expert] the count of the blocks before it, then [experts + expert] of all.
__global__ void __launch_bounds__(kSortThreads) sort_scan_kernel(const int* counts, long long slots, int experts, int blocks,
                                                                 int* position) {
    __shared__ int part[kSortWarps][33];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.x * 32 + lane;
    const int lo = static_cast<int>(static_cast<long long>(blocks) * warp / kSortWarps);
    const int hi = static_cast<int>(static_cast<long long>(blocks) * (warp + 1) / kSortWarps);
    int sum = 0;
    if (e < experts) {
#pragma unroll 8
        for (int b = lo; b < hi; ++b) sum += counts[static_cast<long long>(b) * experts + e];
    }
    part[warp][lane] = sum;
    __syncthreads();
    int run = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        if (w == warp) run = total;
        total += part[w][lane];
    }
    if (e >= experts) return;
#pragma unroll 4
    for (int b = lo; b < hi; ++b) {
        int* to = position + first_slot(slots, b, blocks);
        to[e] = run;
        to[experts + e] = total;
        run += counts[static_cast<long long>(b) * experts + e];
    }
}

// Shared memory: [warp][expert], then per expert the total, the count of the blocks before this
// one, the first row, and 32 words for the scan.
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const ID* ids, long long slots, int experts, int align,
                                                                  int rows, int* offsets, int* position, int* source) {
    extern __shared__ int sm[];
    int* whist = sm;
    int* total = whist + kSortWarps * experts;
    int* before = total + experts;
    int* firsts = before + experts;   // experts + 1
    int* part = firsts + experts + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = gridDim.x;
    // warps of this block that have slots (a few in a serving step: the others' counts are not looked at)
    const long long start = first_slot(slots, blockIdx.x, blocks), end = first_slot(slots, blockIdx.x + 1, blocks);
    const int warps = static_cast<int>((end - start + kPerLane * 32 - 1) / (kPerLane * 32));
    for (int i = threadIdx.x; i < warps * experts; i += kSortThreads) whist[i] = 0;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (blocks > 1) {   // (read before this block's positions are written over it)
        for (int i = threadIdx.x; i < experts; i += kSortThreads) {
            before[i] = position[start + i];
            total[i] = position[start + experts + i];
        }
    } else {
        for (int i = threadIdx.x; i < experts; i += kSortThreads) before[i] = 0;
    }
    __syncthreads();

    // this warp's slots and their counts
    const long long base = start + warp * (kPerLane * 32) + lane;
    int e[kPerLane], rank[kPerLane];
    int* mine = whist + warp * experts;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) e[k] = expert_of(ids, base + k * 32, end, experts);
    if (warp < warps) {
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
            const unsigned same = __match_any_sync(0xffffffffu, e[k]);
            const int ahead = __popc(same & ((1u << lane) - 1u));
            rank[k] = e[k] >= 0 ? mine[e[k]] + ahead : 0;   // among this warp's slots of the expert
            __syncwarp();
            if (e[k] >= 0 && ahead == 0) mine[e[k]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // (a thread per expert: at most kMaxExperts = 1024) counts of the warps before each warp
    const int x = threadIdx.x;
    int length = 0;
    if (x < experts) {
        int run = before[x];
#pragma unroll 8
        for (int w = 0; w < warps; ++w) {
            const int c = whist[w * experts + x];
            whist[w * experts + x] = run;
            run += c;
        }
        if (blocks == 1) total[x] = run;
        length = (total[x] + align - 1) / align * align;
    }
    // first rows: a scan of the rounded lengths
    int inc = length;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int own = part[lane];
        int sum = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += o;
        }
        part[lane] = sum - own;
    }
    __syncthreads();
    inc += part[warp];
    if (x < experts) firsts[x + 1] = inc;
    if (x == 0) firsts[0] = 0;
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i <= experts; i += kSortThreads) offsets[i] = firsts[i];
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        const long long i = base + k * 32;
        if (i >= end) continue;
        int r = -1;
        if (e[k] >= 0) {
            r = firsts[e[k]] + mine[e[k]] + rank[k];
            if (r < rows) source[r] = static_cast<int>(i);
        }
        position[i] = r;
    }
    // rows without a slot: behind each expert's own, and behind the last expert's
    for (int i = blockIdx.x * kSortWarps + warp; i < experts; i += blocks * kSortWarps)
        for (int r = firsts[i] + total[i] + lane; r < min(firsts[i + 1], rows); r += 32) source[r] = -1;
    for (long long r = firsts[experts] + static_cast<long long>(blockIdx.x) * kSortThreads + threadIdx.x; r < rows;
         r += static_cast<long long>(blocks) * kSortThreads)
        source[r] = -1;
}

constexpr int kZeroRows = 16;

// Zeros in those of the rows r0 .. r0+15 that no slot has, this thread's eight columns.
template <typename T, bool VEC>
__device__ __forceinline__ void zero_rows(const int* source, int r0, int rows, T* out, long long ldo, int c, int cols) {
    const float z[8] = {};
    bool none[kZeroRows];   // (all looked up before the first is used)
#pragma unroll
    for (int i = 0; i < kZeroRows; ++i) none[i] = r0 + i < rows && source[r0 + i] < 0;
#pragma unroll
    for (int i = 0; i < kZeroRows; ++i)
        if (none[i]) store_columns<VEC>(out + (r0 + i) * ldo, c, cols, z);
}

// blockIdx.x: a token, or behind the tokens 16 rows to clear; blockIdx.y: a block's share of
// the columns.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) gather_kernel(const RouteRows a) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int c = first_column<VEC>(blockIdx.y * blockDim.x + threadIdx.x);
    if (c >= a.cols) return;
    T* out = static_cast<T*>(a.out);
    if (blockIdx.x >= static_cast<unsigned>(a.tokens)) {
        zero_rows<T, VEC>(a.source, (blockIdx.x - a.tokens) * kZeroRows, a.rows, out, a.ldo, c, a.cols);
        return;
    }
    const long long t = blockIdx.x;
    Raw8<T> raw;
    float v[8];
    load_columns<VEC>(raw, static_cast<const T*>(a.x), t * a.ldx, c, a.cols, true);
    raw.get(v);
    for (int j = 0; j < a.top; ++j) {
        const int r = a.position[t * a.top + j];
        if (r >= 0 && r < a.rows) store_columns<VEC>(out + r * a.ldo, c, a.cols, v);   // (rounding gives v back)
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) combine_kernel(const RouteRows a) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int c = first_column<VEC>(blockIdx.y * blockDim.x + threadIdx.x);
    if (c >= a.cols) return;
    const long long t = blockIdx.x;
    const T* y = static_cast<const T*>(a.x);
    float sum[8] = {};
    // the loads of some slots in flight at a time
    constexpr int N = sizeof(T) == 2 ? 8 : 4;
    for (int j0 = 0; j0 < a.top; j0 += N) {
        Raw8<T> raw[N];
        float w[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int j = j0 + k;
            const int r = j < a.top ? a.position[t * a.top + j] : -1;
            const bool in = r >= 0 && r < a.rows;
            w[k] = in ? (a.weights ? a.weights[t * a.top + j] : 1.0f) : 0.0f;
            load_columns<VEC>(raw[k], y, r * a.ldx, c, a.cols, in);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float v[8];
            raw[k].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[k], v[i], sum[i]);
        }
    }
    store_columns<VEC>(static_cast<T*>(a.out) + t * a.ldo, c, a.cols, sum);
}

// A block per token: its gradient row is read for eight slots at a time. blockIdx.x behind the
// tokens: rows to clear.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) combine_grad_kernel(const RouteRows a) {
    __shared__ float part[8][8];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    T* dy = static_cast<T*>(a.out);
    const int c0 = first_column<VEC>(threadIdx.x);
    if (blockIdx.x >= static_cast<unsigned>(a.tokens)) {
        for (int c = c0; c < a.cols; c += blockDim.x * 8)
            zero_rows<T, VEC>(a.source, (blockIdx.x - a.tokens) * kZeroRows, a.rows, dy, a.ldo, c, a.cols);
        return;
    }
    const long long t = blockIdx.x;
    const T* g = static_cast<const T*>(a.x) + t * a.ldx;
    const T* y = static_cast<const T*>(a.y);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int j0 = 0; j0 < a.top; j0 += 8) {
        int r[8];
        float w[8], dot[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int j = j0 + k;
            r[k] = j < a.top ? a.position[t * a.top + j] : -1;
            if (r[k] >= a.rows) r[k] = -1;
            w[k] = r[k] >= 0 ? (a.weights ? a.weights[t * a.top + j] : 1.0f) : 0.0f;
            dot[k] = 0.0f;
        }
        for (int c = c0; c < a.cols; c += blockDim.x * 8) {
            Raw8<T> raw[8], rawg;
            float gv[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {   // (nothing is read for a dropped slot: zeros)
                const bool in = a.dw && r[k] >= 0;
                load_columns<VEC>(raw[k], y, r[k] * a.ldy, c, a.cols, in);
            }
            load_columns<VEC>(rawg, g, 0, c, a.cols, true);
            rawg.get(gv);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float v[8];
                raw[k].get(v);
                if (r[k] >= 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[k] = fmaf(gv[i], v[i], dot[k]);
                }
                if (dy && r[k] >= 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = w[k] * gv[i];
                    store_columns<VEC>(dy + r[k] * a.ldo, c, a.cols, v);
                }
            }
        }
        if (!a.dw) continue;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], d);
            if (lane == 0) part[warp][k] = dot[k];
        }
        __syncthreads();
        if (threadIdx.x < 8 && j0 + threadIdx.x < a.top) {
            float sum = 0.0f;
            for (int i = 0; i < warps; ++i) sum += part[i][threadIdx.x];
            a.dw[t * a.top + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

template <typename T>
bool vec16(const void* p, long long ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * static_cast<long long>(sizeof(T)) % 16 == 0;
}

int row_threads(int cols) { return std::min(256, ((cols + 7) / 8 + 31) / 32 * 32); }

template <typename T>
cudaError_t gather(const RouteRows& a, cudaStream_t stream) {
    const int th = row_threads(a.cols);
    const long long x = static_cast<long long>(a.tokens) + (a.rows + kZeroRows - 1) / kZeroRows;
    if (x == 0) return cudaSuccess;
    const int by = (a.cols + th * 8 - 1) / (th * 8);
    if (x > 0x7fffffffll || by > 65535) return cudaErrorInvalidValue;
    const bool vec = vec16<T>(a.x, a.ldx) && vec16<T>(a.out, a.ldo);
    return launch_pdl(vec ? gather_kernel<T, true> : gather_kernel<T, false>, dim3(static_cast<unsigned>(x), by), th, 0,
                      stream, a);
}

template <typename T>
cudaError_t combine(const RouteRows& a, cudaStream_t stream) {
    if (a.tokens == 0) return cudaSuccess;
    const int th = row_threads(a.cols);
    const int by = (a.cols + th * 8 - 1) / (th * 8);
    if (by > 65535) return cudaErrorInvalidValue;
    const bool vec = vec16<T>(a.x, a.ldx) && vec16<T>(a.out, a.ldo);
    return launch_pdl(vec ? combine_kernel<T, true> : combine_kernel<T, false>, dim3(a.tokens, by), th, 0, stream, a);
}

template <typename T>
cudaError_t combine_grad(const RouteRows& a, cudaStream_t stream) {
    const long long x = static_cast<long long>(a.tokens) + (a.out ? (a.rows + kZeroRows - 1) / kZeroRows : 0);
    if (x == 0) return cudaSuccess;
    if (x > 0x7fffffffll) return cudaErrorInvalidValue;
    const bool vec = vec16<T>(a.x, a.ldx) && (!a.dw || vec16<T>(a.y, a.ldy)) && (!a.out || vec16<T>(a.out, a.ldo));
    return launch_pdl(vec ? combine_grad_kernel<T, true> : combine_grad_kernel<T, false>, dim3(static_cast<unsigned>(x)),
                      row_threads(a.cols), 0, stream, a);
}

// (what a block of the sort needs of shared memory for the most experts)
constexpr size_t sort_smem(int experts) { return sizeof(int) * ((kSortWarps + 3) * static_cast<size_t>(experts) + 1 + kSortWarps); }

template <typename ID>
cudaError_t sort(long long slots, const ID* ids, int experts, int align, int rows, int* offsets, int* position,
                 int* source, cudaStream_t stream) {
    const int blocks = static_cast<int>(std::max(1ll, (slots + kSortChunk - 1) / kSortChunk));
    const size_t smem = sort_smem(experts);
    if (smem > 48 * 1024) {   // (the same limit each time: threads that set it do not get in each other's way)
        const cudaError_t err = cudaFuncSetAttribute(sort_place_kernel<ID>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(sort_smem(kMaxExperts)));
        if (err != cudaSuccess) return err;
    }
    if (blocks > 1) {
        // (blocks * experts counts: at most (slots / 4096 + 1) * 1024, less than the slots and so than the rows)
        cudaError_t err = launch_pdl(sort_count_kernel<ID>, dim3(blocks), kSortThreads, sizeof(int) * experts, stream, ids,
                                     slots, experts, source);
        if (err != cudaSuccess) return err;
        err = launch_pdl(sort_scan_kernel, dim3((experts + 31) / 32), kSortThreads, 0, stream, source, slots, experts, blocks,
                         position);
        if (err != cudaSuccess) return err;
    }
    return launch_pdl(sort_place_kernel<ID>, dim3(blocks), kSortThreads, smem, stream, ids, slots, experts, align, rows,
                      offsets, position, source);
}

}  // namespace

cudaError_t launch_sort(long long slots, const void* ids, int id_bytes, int experts, int align, int rows, int* offsets,
                        int* position, int* source, cudaStream_t stream) {
    if (id_bytes == 8)
        return sort(slots, static_cast<const long long*>(ids), experts, align, rows, offsets, position, source, stream);
    return sort(slots, static_cast<const int*>(ids), experts, align, rows, offsets, position, source, stream);
}

cudaError_t launch_gather(const RouteRows& a, cudaStream_t stream) {
    return a.f32 ? gather<float>(a, stream) : gather<__nv_bfloat16>(a, stream);
}

cudaError_t launch_combine(const RouteRows& a, cudaStream_t stream) {
    return a.f32 ? combine<float>(a, stream) : combine<__nv_bfloat16>(a, stream);
}

cudaError_t launch_combine_grad(const RouteRows& a, cudaStream_t stream) {
    return a.f32 ? combine_grad<float>(a, stream) : combine_grad<__nv_bfloat16>(a, stream);
}

}  // namespace tcl
