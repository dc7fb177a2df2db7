// Eight neighbouring values of a row at a time, as fp32: the piece one thread handles in
// the kernels that stream rows (quantising, gathering, combining).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace tcl {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Eight values as they lie in memory: loaded first, widened where they are used, so that many
// loads can be in flight without as many fp32 registers.
template <typename T>
struct Raw8;

template <>
struct __align__(16) Raw8<__nv_bfloat16> {
    uint4 u;
    // values p[0..n) (n may be past 8, or below 1), the rest zeros; vec: p is 16-byte aligned
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int n, bool vec) {
        if (vec && n >= 8) {
            u = *reinterpret_cast<const uint4*>(p);
            return;
        }
        uint32_t w[4] = {0, 0, 0, 0};
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i / 2] |= static_cast<uint32_t>(h[i]) << (16 * (i & 1));
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { unpack8(u, v); }
};

template <>
struct __align__(16) Raw8<float> {
    float f[8];
    __device__ __forceinline__ void load(const float* p, int n, bool vec) {
        if (vec && n >= 8) {
            const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? p[i] : 0.0f;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i];
    }
};

// A row's columns are dealt out to threads, eight each. Where rows start on 16 bytes (VEC) a
// thread takes neighbouring ones, its first being first_column; elsewhere every 32nd, so that a
// warp's single-element accesses are to neighbours (neighbours to a thread there took four times
// as long).
template <bool VEC>
__device__ __forceinline__ int first_column(int thread) {
    return VEC ? thread * 8 : (thread & ~31) * 8 + (thread & 31);
}

// The columns of the row at base + at (in = false: zeros, and nothing is read).
template <bool VEC, typename T>
__device__ __forceinline__ void load_columns(Raw8<T>& r, const T* base, long long at, int c, int cols, bool in) {
    if constexpr (VEC) {
        r.load(base + (in ? at + c : 0ll), in ? cols - c : 0, true);
    } else {
        const T* row = base + (in ? at : 0ll);
        if (!in) cols = 0;
        alignas(16) T v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + 32 * i < cols ? row[c + 32 * i] : T(0.0f);
        r = *reinterpret_cast<const Raw8<T>*>(v);
    }
}

// (each value rounded once, to nearest even)
__device__ __forceinline__ __nv_bfloat16 as_type(float v, __nv_bfloat16) { return __float2bfloat16_rn(v); }
__device__ __forceinline__ float as_type(float v, float) { return v; }

template <bool VEC, typename T>
__device__ __forceinline__ void store_columns(T* row, int c, int cols, const float (&v)[8]) {
    if (VEC && c + 8 <= cols) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(row + c) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                            pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        } else {
            reinterpret_cast<float4*>(row + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(row + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = c + (VEC ? i : 32 * i);
        if (k < cols) row[k] = as_type(v[i], T());
    }
}

}  // namespace tcl
