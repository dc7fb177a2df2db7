// The norm over many tensors of gradients, and their scaling down to a bound on it.
//
// What bounds both is the memory: one pass reads every gradient, another reads and writes it. The
// tensors' addresses travel in the launch's parameters (no copy to the GPU, so that a captured
// launch replays on its own), their elements are dealt out in pieces over all
// tensors, and a block finds a piece's tensor by bisection. The second pass walks the pieces
// backwards: what the first one read last is still in L2. A thread has 64 bytes in flight in the first pass,
// 128 in the second: 10^9 bf16 values in 0.28 ms (7.1 TB/s) and 0.61 ms (6.5 TB/s read and written;
// 5.5 with 64 bytes and half of the blocks).
//
// Squares are added in fp32 within a thread's 32 elements and in fp64 from there on, in an order
// that depends on the lengths and on the addresses modulo 16 (which elements make up a thread's 32): the same
// tensors give the same norm, equal values at another alignment may give its neighbour. Where 32 squares leave
// fp32's range (elements beyond 2^63 or all below 2^-50), they are added again in fp64.
//
// The factor is rounded to fp32, its product with a value to fp32 and then to the type: an fp32 result is off by two half
// steps instead of one, a bf16 one by 2^-15 of a step more than a half. A factor in two parts, and a second
// multiplication for each value, would spare that.
#include <cuda_bf16.h>

#include "clip_launch.cuh"
#include "fp8_launch.cuh"

namespace tcl {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int tensor_of(const ClipTensors& a, long long piece) {
    int lo = 0, hi = a.n - 1;   // the last tensor that starts at or before the piece (empty ones have none)
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.t[mid].before <= piece)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Elements before the next 16-byte unit.
template <typename T>
__device__ __forceinline__ int to_unit(const T* p) {
    return static_cast<int>(-reinterpret_cast<uintptr_t>(p) & 15) / static_cast<int>(sizeof(T));
}

template <typename T>
__device__ __forceinline__ float value(T x);
template <>
__device__ __forceinline__ float value(float x) { return x; }
template <>
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ void unpack(uint4 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// The sum over a block of 256, in its first warp alone; its order is fixed. (An SM has two fp64 lanes: an instruction
// of eight warps takes 128 cycles.)
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double sh[kThreads];
    sh[threadIdx.x] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x < 32) {
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) s += sh[32 * i + threadIdx.x];
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    }
    return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 5) square_sums_kernel(const __grid_constant__ ClipTensors a, double* parts) {
    constexpr int U = 16 / sizeof(T), Q = 32 / U;   // elements of a 16-byte unit, units of a thread's 32 elements
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    double sum = 0.0;
    auto squares = [&](auto& v) {   // of some units
        float s = 0.0f;
        uint32_t any = 0;
#pragma unroll
        for (auto& w : v) {
            float f[U];
            unpack(w, f);
#pragma unroll
            for (int i = 0; i < U; ++i) s = fmaf(f[i], f[i], s);
            any |= w.x | w.y | w.z | w.w;
        }
        if (s >= 7.9e-31f && s < __int_as_float(0x7f800000)) {   // 2^-100, infinity
            sum += static_cast<double>(s);
        } else if (any) {
#pragma unroll
            for (auto& w : v) {
                float f[U];
                unpack(w, f);
#pragma unroll
                for (int i = 0; i < U; ++i) sum += static_cast<double>(f[i]) * f[i];
            }
        }
    };
    for (long long piece = blockIdx.x; piece < a.pieces; piece += gridDim.x) {
        const ClipTensor& t = a.t[tensor_of(a, piece)];
        const long long at = (piece - t.before) * a.piece;
        const T* x = static_cast<const T*>(t.from) + at;
        int n = static_cast<int>(t.n - at < a.piece ? t.n - at : a.piece);
        const int lead = min(n, to_unit(x));
        if (threadIdx.x < lead) {
            const double f = value(x[threadIdx.x]);
            sum += f * f;
        }
        x += lead;
        n -= lead;
        int done = 0;
        {
            constexpr int STEP = kThreads * 32;
            const uint4* x4 = reinterpret_cast<const uint4*>(x);
            for (; done + STEP <= n; done += STEP) {
                uint4 v[Q];
#pragma unroll
                for (int q = 0; q < Q; ++q) v[q] = x4[done / U + q * kThreads + threadIdx.x];
                squares(v);
            }
            for (int i = done / U + threadIdx.x; i < n / U; i += kThreads) {
                const uint4 v[1] = {x4[i]};
                squares(v);
            }
            done = n / U * U;
        }
        for (int i = done + threadIdx.x; i < n; i += kThreads) {
            const double f = value(x[i]);
            sum += f * f;
        }
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

// The norm, in the block's first warp alone.
__device__ __forceinline__ double norm_of(const double* parts, int n) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += parts[i];
    s = block_sum(s);
    return threadIdx.x < 32 ? sqrt(s) : 0.0;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* parts, int n, float* norm) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const double v = norm_of(parts, n);
    if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ ClipTensors a, const double* parts, int nparts,
                                                        float bound, float* norm) {
    constexpr int U = 16 / sizeof(T), Q = 8;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    __shared__ float sh[3];
    const double length = norm_of(parts, nparts);
    if (threadIdx.x == 0) {
        const float told = static_cast<float>(length);
        if (norm && blockIdx.x == 0) *norm = told;
        // (a norm that is NaN or infinite, in fp32, scales nothing: the caller, who is told of it, drops the step)
        const bool larger = length > bound && told < __int_as_float(0x7f800000);
        // A factor below fp32's normal numbers keeps its digits: 2^-126 of it goes first. (What that takes from a
        // small element is less than half of fp32's smallest number times the rest, and that is below 1.)
        const double factor = larger ? static_cast<double>(bound) / length : 1.0;
        const bool tiny = factor < 0x1p-126;
        sh[0] = larger ? 1.0f : 0.0f;
        sh[1] = tiny ? 0x1p-126f : 1.0f;
        sh[2] = static_cast<float>(tiny ? factor * 0x1p126 : factor);
    }
    __syncthreads();
    const bool scaled = sh[0] != 0.0f;
    const float first = sh[1], f = sh[2];
    for (long long back = blockIdx.x; back < a.pieces; back += gridDim.x) {
        const long long piece = a.pieces - 1 - back;
        const ClipTensor& t = a.t[tensor_of(a, piece)];
        if (!scaled && t.from == t.to) continue;
        const long long at = (piece - t.before) * a.piece;
        const T* x = static_cast<const T*>(t.from) + at;
        T* y = static_cast<T*>(t.to) + at;
        int n = static_cast<int>(t.n - at < a.piece ? t.n - at : a.piece);
        int done = 0;
        if ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) % 16 == 0) {
            const int lead = min(n, to_unit(x));
            if (threadIdx.x < lead) y[threadIdx.x] = scaled ? static_cast<T>(value(x[threadIdx.x]) * first * f) : x[threadIdx.x];
            x += lead;
            y += lead;
            n -= lead;
            constexpr int STEP = kThreads * Q * U;
            const uint4* x4 = reinterpret_cast<const uint4*>(x);
            uint4* y4 = reinterpret_cast<uint4*>(y);
            auto times = [&](uint4 v) {
                float e[U];
                unpack(v, e);
#pragma unroll
                for (int i = 0; i < U; ++i) e[i] = e[i] * first * f;
                return scaled ? pack(e) : v;
            };
            for (; done + STEP <= n; done += STEP) {
                uint4 v[Q];
#pragma unroll
                for (int q = 0; q < Q; ++q) v[q] = x4[done / U + q * kThreads + threadIdx.x];
#pragma unroll
                for (int q = 0; q < Q; ++q) __stcs(y4 + done / U + q * kThreads + threadIdx.x, times(v[q]));
            }
            for (int i = done / U + threadIdx.x; i < n / U; i += kThreads) y4[i] = times(x4[i]);
            done = n / U * U;
        }
        for (int i = done + threadIdx.x; i < n; i += kThreads) y[i] = scaled ? static_cast<T>(value(x[i]) * first * f) : x[i];
    }
}

}  // namespace

int clip_blocks(long long pieces) { return static_cast<int>(pieces < 1 ? 1 : pieces > kClipBlocks ? kClipBlocks : pieces); }

cudaError_t launch_square_sums(const ClipTensors& a, double* parts, cudaStream_t stream) {
    return launch_pdl(a.f32 ? square_sums_kernel<float> : square_sums_kernel<__nv_bfloat16>, dim3(clip_blocks(a.pieces)),
                      kThreads, 0, stream, a, parts);
}

cudaError_t launch_norm(const double* parts, int n, float* norm, cudaStream_t stream) {
    return launch_pdl(norm_kernel, dim3(1), kThreads, 0, stream, parts, n, norm);
}

cudaError_t launch_clip(const ClipTensors& a, const double* parts, int n, float bound, float* norm, cudaStream_t stream) {
    return launch_pdl(a.f32 ? clip_kernel<float> : clip_kernel<__nv_bfloat16>, dim3(clip_blocks(a.pieces)), kThreads, 0,
                      stream, a, parts, n, bound, norm);
}

}  // namespace tcl
