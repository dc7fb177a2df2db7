// Quantising to e4m3 with one fp32 scale for each 128 values.
//
//   s = max(max|x| / 448, 2^-126),  q = e4m3(x · (1/s)), rounded to nearest even
//
// One division for each group and one product for each value. The largest magnitude is
// taken over the values' bit patterns without their sign, whose order is that of the
// magnitudes with infinities and NaN above all numbers, so a NaN or an infinity reaches
// the scale. They read X once and write Q once and are bound by memory (16384 × 4096 bf16, floor 30 us:
// down columns 39 us, blocks 34, transposed 36; fp32, floor 50: 53, 51, 51; 64 fp32 matrices of
// 2048 × 1024, floor 99: 96, some of it still in the L2), but for bf16 along rows: 41 us, 4.9 TB/s, 79 % of
// the issue slots busy with 38 M warp instructions where blocks take 24 M (addresses, bounds and
// reductions for each group of 128 values instead of each 128 × 128); fp32 along rows 52.
#include <cuda_fp8.h>

#include <algorithm>

#include "fp8_launch.cuh"
#include "rows8.cuh"

namespace tcl {
namespace {

constexpr int kG = 128;

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// (a NaN has to come through the lower bound of the scale: fmaxf would drop it)
__device__ __forceinline__ float group_scale(uint32_t top) {
    const float s = __fdiv_rn(__uint_as_float(top), 448.0f);
    const float least = 1.17549435e-38f;   // 2^-126
    return s < least ? least : s;
}

__device__ __forceinline__ uint2 quant8(const float (&v)[8], float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv), __NV_SATFINITE,
                                                     __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv),
                                                     __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

// The first n of the 8 bytes, and zeros behind them (behind the matrix' end) where the row has room
// for them. (The zeros are put in here: those loaded there times the reciprocal of a NaN's scale are
// not zeros. Off the whole pieces' path.)
__device__ __forceinline__ void put8(uint8_t* p, int n, int room, bool vec, uint2 w) {
    if (vec && n >= 8) {
        *reinterpret_cast<uint2*>(p) = w;
        return;
    }
    const uint64_t kept = (static_cast<uint64_t>(w.y) << 32 | w.x) & (n >= 8 ? ~0ull : n > 0 ? (1ull << (8 * n)) - 1 : 0ull);
    if (vec && room >= 8) {
        *reinterpret_cast<uint64_t*>(p) = kept;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < room) p[i] = static_cast<uint8_t>(kept >> (8 * i));
}

// Groups along the rows: sixteen lanes (a team) hold a group, eight values each. A block's
// eight teams take neighbouring groups, of one row or, where a row has fewer than eight, of
// several (`row_teams`, a power of two, to a row), and N rows one after another whose loads
// are all issued first. With an order, a token's row is read and quantised once and written to
// each of its rows; blocks behind the tokens' write the rows that no token has.
constexpr int kTeams = 8, kZeroRows = 32;

// (blocks an SM: with nine of bf16 and N = 4, for three more registers, 16384 × 4096 took 43 us; with
// seven of fp32 53 instead of 51)
template <typename T, int N>
__global__ void __launch_bounds__(16 * kTeams, N == 1 ? 12 : sizeof(T) == 2 ? 10 : 8)
    quant_rows_kernel(const QuantRows a, int groups, int row_teams_log2, int quant_blocks, int wcols, bool vec_in, bool vec_out) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int team = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int row_teams = 1 << row_teams_log2, rows_at_once = kTeams >> row_teams_log2;
    if (blockIdx.x >= quant_blocks) {
        if (blockIdx.y > 0) return;
        const int r0 = (blockIdx.x - quant_blocks) * kZeroRows;
        for (int r = r0 + team; r < min(r0 + kZeroRows, a.out_rows); r += kTeams) {
            if (a.source[r] >= 0) continue;
            for (int c = l * 8; c < wcols; c += 128) put8(a.q + r * a.ldq + c, a.cols - c, wcols - c, vec_out, make_uint2(0u, 0u));
            for (int g = l; g < groups; g += 16) a.scale[r * a.s_row + g * a.s_group] = group_scale(0u);
        }
        return;
    }
    const int g = blockIdx.y * row_teams + (team & (row_teams - 1));
    const int row0 = blockIdx.x * (N * rows_at_once) + (team >> row_teams_log2);
    const int c = g * kG + l * 8;
    Raw8<T> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = row0 + i * rows_at_once;
        const bool in = row < a.rows && g < groups;
        raw[i].load(static_cast<const T*>(a.x) + (in ? row * a.ldx + c : 0), in ? a.cols - c : 0, vec_in);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = row0 + i * rows_at_once;
        float v[8];
        raw[i].get(v);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, magnitude(v[j]));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (row >= a.rows || g >= groups) continue;   // (uniform over the team)
        const float s = group_scale(top);
        const uint2 w = quant8(v, __frcp_rn(s));
        for (int j = 0; j < (a.position ? a.top : 1); ++j) {
            const int r = a.position ? a.position[static_cast<long long>(row) * a.top + j] : row;
            if (r < 0 || (a.position && r >= a.out_rows)) continue;
            put8(a.q + r * a.ldq + c, a.cols - c, wcols - c, vec_out, w);
            if (l == 0) a.scale[r * a.s_row + g * a.s_group] = s;
        }
    }
}

// Tiles of 128 × 128 values, 256 threads with eight rows × eight columns each. Transposed
// results go through shared memory, column by column of X as 128 bytes, in pieces of 8 bytes
// whose place is permuted by the column so that neither side has bank conflicts.
// (fp32 without a bound took 92 registers, two blocks an SM: columns 63 us instead of 53; with it blocks
// spill 20 bytes and take 51 us, the floor 50)
template <typename T, QuantTile KIND>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 3 : 4) quant_tiles_kernel(const QuantTiles a, bool vec_in, bool vec_out) {
    constexpr bool TR = KIND != QuantTile::BLOCKS;
    __shared__ uint32_t red[16][kG];
    __shared__ float sc[kG];
    __shared__ uint2 turn[TR ? kG * 16 : 1];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int c0 = blockIdx.x * kG, r0 = blockIdx.y * kG;
    const int c = c0 + cg * 8;
    const T* x = static_cast<const T*>(a.x) + blockIdx.z * a.x_batch;
    Raw8<T> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        int r = r0 + rg * 8 + i;
        bool in = r < a.rows;
        if (KIND == QuantTile::COLUMNS && a.source && in) {
            const int slot = a.source[r];
            r = slot / a.top;
            in = slot >= 0 && r < a.x_rows;
        }
        raw[i].load(x + (in ? r * a.ldx + c : 0), in ? a.cols - c : 0, vec_in);
    }
    uint32_t top[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        raw[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) top[j] = max(top[j], magnitude(v[j]));
    }
    float inv[8];
    if constexpr (KIND == QuantTile::COLUMNS) {
#pragma unroll
        for (int j = 0; j < 8; ++j) red[rg][cg * 8 + j] = top[j];
        __syncthreads();
        if (threadIdx.x < kG) {
            uint32_t t = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) t = max(t, red[i][threadIdx.x]);
            const float s = group_scale(t);
            if (c0 + threadIdx.x < a.cols) a.scale[(c0 + threadIdx.x) * a.s_row + blockIdx.y * a.s_group] = s;
            sc[threadIdx.x] = __frcp_rn(s);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) inv[j] = sc[cg * 8 + j];
    } else {
        uint32_t t = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) t = max(t, top[j]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, d));
        if ((threadIdx.x & 31) == 0) red[0][threadIdx.x >> 5] = t;
        __syncthreads();
        t = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) t = max(t, red[0][i]);
        const float s = group_scale(t);
        if (threadIdx.x == 0) {
            const unsigned r = KIND == QuantTile::BLOCKS ? blockIdx.y : blockIdx.x;
            const unsigned g = KIND == QuantTile::BLOCKS ? blockIdx.x : blockIdx.y;
            a.scale[blockIdx.z * a.s_batch + r * a.s_row + g * a.s_group] = s;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) inv[j] = __frcp_rn(s);
    }
    uint8_t* q = a.q + blockIdx.z * a.q_batch;
    if constexpr (!TR) {
        const int wcols = static_cast<int>(min(a.room, static_cast<long long>((a.cols + 15) & ~15)));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + rg * 8 + i;
            float v[8];
            raw[i].get(v);
            if (r < a.rows && c < wcols) put8(q + r * a.ldq + c, a.cols - c, wcols - c, vec_out, quant8(v, inv[0]));
        }
        return;
    }
    if constexpr (TR) {
        float v[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i].get(v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = v[i][j];
            turn[(cg * 8 + j) * 16 + (rg ^ cg)] = quant8(w, inv[j]);
        }
        __syncthreads();
        const int wrows = static_cast<int>(min(a.room, static_cast<long long>((a.rows + 15) & ~15)));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int cc = k * 16 + rg, r = r0 + cg * 8;   // sixteen threads write a column's 128 bytes
            if (c0 + cc < a.cols && r < wrows)
                put8(q + (c0 + cc) * a.ldq + r, a.rows - r, wrows - r, vec_out, turn[cc * 16 + (cg ^ (cc >> 3))]);
        }
    }
}

__global__ void __launch_bounds__(256) copy_bytes_kernel(const uint8_t* src, long long ld, long long batch_stride,
                                                         uint8_t* dst, long long ld_dst, int rows, int cols) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    src += blockIdx.z * batch_stride;
    dst += static_cast<long long>(blockIdx.z) * rows * ld_dst;
    const int c = blockIdx.x * 256 + threadIdx.x;   // (the grid covers the columns: a step past them could pass 32 bits)
    if (c >= cols) return;
    for (int r = blockIdx.y; r < rows; r += gridDim.y) dst[r * ld_dst + c] = src[r * ld + c];
}

template <typename T>
bool row_aligned(const void* p, long long ld, int bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * static_cast<long long>(sizeof(T)) % bytes == 0;
}

template <typename T, int N>
cudaError_t quant_rows_n(const QuantRows& a, int groups, int row_teams_log2, cudaStream_t stream) {
    const int rows_at_once = kTeams >> row_teams_log2;
    const long long blocks = (static_cast<long long>(a.rows) + N * rows_at_once - 1) / (N * rows_at_once);
    const long long zero = a.position ? (a.out_rows + kZeroRows - 1) / kZeroRows : 0;
    const int by = (groups + (1 << row_teams_log2) - 1) >> row_teams_log2;
    if (blocks + zero > 0x7fffffffll || by > 65535) return cudaErrorInvalidValue;
    if (blocks + zero == 0) return cudaSuccess;
    const int wcols = static_cast<int>(std::min<long long>(a.ldq, (a.cols + 15) & ~15));
    return launch_pdl(quant_rows_kernel<T, N>, dim3(static_cast<unsigned>(blocks + zero), by), 16 * kTeams, 0, stream, a,
                      groups, row_teams_log2, static_cast<int>(blocks), wcols, row_aligned<T>(a.x, a.ldx, 16),
                      row_aligned<uint8_t>(a.q, a.ldq, 8));
}

template <typename T>
cudaError_t quant_rows(const QuantRows& a, cudaStream_t stream) {
    const int groups = (a.cols + kG - 1) / kG;
    int log2 = 0;
    while (log2 < 3 && (1 << log2) < groups) ++log2;
    // four rows per thread where that leaves enough blocks to fill the GPU several times over
    if (static_cast<long long>(a.rows) * groups >= 4ll * kTeams * 4096)
        return quant_rows_n<T, 4>(a, groups, log2, stream);
    return quant_rows_n<T, 1>(a, groups, log2, stream);
}

// One launch for each 65,535 rows of tiles and 65,535 matrices: what the grid's axes hold.
template <typename T, QuantTile KIND>
cudaError_t quant_tiles(const QuantTiles& a, cudaStream_t stream) {
    constexpr int kAxis = 65535;
    const bool vec_in = row_aligned<T>(a.x, a.ldx, 16) && (a.batch < 2 || a.x_batch * sizeof(T) % 16 == 0);
    const bool vec_out = row_aligned<uint8_t>(a.q, a.ldq, 8) && (a.batch < 2 || a.q_batch % 8 == 0);
    const long long rows = a.rows;
    for (long long z = 0; z < a.batch; z += kAxis)
        for (long long r = 0; r < rows; r += kAxis * kG) {
            QuantTiles p = a;
            p.batch = static_cast<int>(std::min<long long>(a.batch - z, kAxis));
            p.rows = static_cast<int>(std::min<long long>(rows - r, kAxis * kG));
            p.room = KIND == QuantTile::BLOCKS ? a.ldq : a.ldq - r;
            p.q += z * a.q_batch + (KIND == QuantTile::BLOCKS ? r * a.ldq : r);
            p.scale += z * a.s_batch + r / kG * (KIND == QuantTile::BLOCKS ? a.s_row : a.s_group);
            if (a.source)
                p.source += r;   // (its rows are X's whichever they are)
            else
                p.x = static_cast<const T*>(a.x) + z * a.x_batch + r * a.ldx;
            const dim3 grid((p.cols + kG - 1) / kG, (p.rows + kG - 1) / kG, p.batch);
            const cudaError_t err = launch_pdl(quant_tiles_kernel<T, KIND>, grid, 256, 0, stream, p, vec_in, vec_out);
            if (err != cudaSuccess) return err;
        }
    return cudaSuccess;
}

template <typename T>
cudaError_t quant_tiles_of(QuantTile kind, const QuantTiles& a, cudaStream_t stream) {
    switch (kind) {
        case QuantTile::COLUMNS: return quant_tiles<T, QuantTile::COLUMNS>(a, stream);
        case QuantTile::BLOCKS: return quant_tiles<T, QuantTile::BLOCKS>(a, stream);
        default: return quant_tiles<T, QuantTile::BLOCKS_T>(a, stream);
    }
}

}  // namespace

cudaError_t launch_quant_rows(const QuantRows& a, cudaStream_t stream) {
    return a.f32 ? quant_rows<float>(a, stream) : quant_rows<__nv_bfloat16>(a, stream);
}

cudaError_t launch_quant_tiles(QuantTile kind, const QuantTiles& a, cudaStream_t stream) {
    return a.f32 ? quant_tiles_of<float>(kind, a, stream) : quant_tiles_of<__nv_bfloat16>(kind, a, stream);
}

cudaError_t launch_copy_bytes(const uint8_t* src, long long ld, long long batch_stride, uint8_t* dst, long long ld_dst,
                              int batch, int rows, int cols, cudaStream_t stream) {
    if (batch < 1 || rows < 1) return cudaSuccess;
    const dim3 grid((cols + 255) / 256, std::min(rows, 4096), batch);
    return launch_pdl(copy_bytes_kernel, grid, 256, 0, stream, src, ld, batch_stride, dst, ld_dst, rows, cols);
}

}  // namespace tcl
