// Products of bf16 matrices, D = A·B^T (M × N, sums in fp32), with what a model does next in the
// same kernel: a 256 × 256 tile on a pair of SMs (tcgen05.mma.cta_group::2).
//
// Either operand may be stored with K contiguous (rows of K) or with its rows contiguous
// (K rows of M or N values): a layer's product reads both as they are stored, its gradients read
// one or both of the same buffers along the other axis, and nothing is ever transposed in memory.
//
// The ends (DenseEnd):
//   STORE      D, times a factor for each row, plus an fp32 matrix, as bf16 or fp32. K may be cut
//              into `splits` ranges, whose fp32 sums go to a workspace and are joined in their
//              order by another kernel. K may run over two operand pairs, one after the other
//              (dx = dgate·Wgate + dup·Wup as one product).
//   GATE       the columns of B are 128 rows of one matrix and 128 of another (each SM of a pair
//              loads one of them), so that a thread finds a gate and its partner in the same
//              row of tensor memory: h = act(gate)·up, and gate and up in bf16 where a backward
//              pass will want them
//   GATE_GRAD  D = dh; dgate = dh·up·act'(gate), dup = dh·act(gate)
//   ENTROPY    D = logits: for each row the sum of the exponentials over 128 columns, the target's
//              logit, and in training the exponentials themselves in bf16 (dense_entropy.cuh says
//              what they are relative to)
//
// Roles of each CTA: warp 0 loads (TMA, 128-byte swizzle, a ring of 64-value k-blocks), warp 1 of
// the pair's leader issues the MMAs into one of two accumulators in tensor memory, warps 2 to 9
// read the other one (each 32 lanes × half of the columns) and store through slabs of 32 rows ×
// 128 bytes, copied out by the tensor copy engine. A pair walks its tiles blockIdx/2, + pairs, ...
//
// Every wait is bounded; a role that gives up raises the pair's abort flag.
#pragma once

#include "gemm_kernel_pair.cuh"
#include "rows8.cuh"

namespace tcl {

enum class DenseEnd : int { STORE, GATE, GATE_GRAD, ENTROPY };
enum : int { DENSE_SILU = 0, DENSE_GELU = 1, DENSE_GELU_TANH = 2 };

struct DenseOut {
    void* p;
    long long ld;     // elements
    int cols;         // columns that may be written (a buffer of this library's own: whole 16-byte pieces)
    int tma;          // rows start on 16-byte pieces: there is a tensor map
};

struct DenseParams {
    int M, N;              // rows and columns of D (GATE: N columns of h)
    int kb0, kb1;          // k-blocks of the first and of the second operand pair (0: one pair)
    int tiles_m, tiles_n, splits, group;
    int f32;               // STORE: fp32 result
    int act;
    DenseOut out[3];       // D, h or dgate or the exponentials; gate or dup; up
    const float* factor;   // STORE: of each row (NULL: ones); a row whose factor is zero is zeros
    const float* plus;     // STORE: added to the result (NULL: nothing)
    long long ld_plus;
    const __nv_bfloat16 *gate, *up;   // GATE_GRAD; rows on 16-byte pieces
    long long ld_kept;
    const void* targets;   // ENTROPY: M of them, int32 or int64
    int wide_targets;
    float2* parts;         // ENTROPY: [128-column chunk][row of D]: exponent taken out, sum
    float* target_logit;   // ENTROPY: [row of D]
    int exps;              // ENTROPY: store the exponentials
    unsigned long long timeout_ns;
    unsigned int* status;
};

// act(g), and its derivative where it is asked for.
template <bool SLOPE>
__device__ __forceinline__ float dense_act(int act, float g, float& slope) {
    if (act == DENSE_GELU) {
        const float p = 0.5f * erfcf(-0.70710678118654752f * g);   // (no cancellation for g < 0)
        if (SLOPE) slope = p + g * 0.39894228040143268f * __expf(-0.5f * g * g);
        return g * p;
    }
    float z = g;
    if (act == DENSE_GELU_TANH) z = 1.5957691216057308f * g * (1.0f + 0.044715f * g * g);   // (1 + tanh(z/2))/2 is the sigmoid of z
    const float s = __fdividef(1.0f, 1.0f + __expf(-z));
    if (SLOPE) {
        if (act == DENSE_GELU_TANH) {
            const float c = fminf(fmaxf(g, -1e4f), 1e4f);   // (s(1 - s) is zero long before that)
            slope = s + c * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 3.0f * 0.044715f * c * c);
        } else {
            slope = s * (1.0f + g * (1.0f - s));
        }
    }
    return g * s;
}

struct DenseCfg {
    static constexpr int BM = 256, BN = 256, BK = 64;
    static constexpr int STAGES = 5;
    static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;   // a CTA's share of a k-block
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EW = 8;                    // epilogue warps
    static constexpr int SLABS = 2, SLAB_BYTES = 32 * 128;
    static constexpr int NBARS = 2 * STAGES + 5;
    static constexpr int THREADS = 64 + 32 * EW;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EW * SLABS * SLAB_BYTES + (NBARS + 2) * 8;
    static_assert(SMEM_BYTES <= 232448, "exceeds the 227 KB per-block shared memory limit");
};

struct DenseUnit {
    int m0, n, z, lo, hi;   // first row, tile column, K range's number and k-blocks
};

__device__ __forceinline__ DenseUnit dense_unit(const DenseParams& p, int u) {
    // `group` tile rows share a pass over the tile columns, so that a wave of the GPU reads few
    // operand rows of either side
    const int tiles = p.tiles_m * p.tiles_n, z = u / tiles, t = u - z * tiles;
    const int g = t / (p.group * p.tiles_n) * p.group, gn = min(p.group, p.tiles_m - g), r = t - g * p.tiles_n;
    const long long kb = p.kb0 + p.kb1;
    DenseUnit U;
    U.m0 = (g + r % gn) * DenseCfg::BM;
    U.n = r / gn;
    U.z = z;
    U.lo = static_cast<int>(kb * z / p.splits);
    U.hi = static_cast<int>(kb * (z + 1) / p.splits);
    return U;
}

// A warp's staging slabs, taken in turn: 32 rows (a lane each) of 128 bytes, 16-byte units
// permuted by the row as the tensor copies do.
struct DenseSlabs {
    uint8_t* base;
    int used, lane;
    __device__ __forceinline__ uint8_t* take() {
        uint8_t* s = base + used * DenseCfg::SLAB_BYTES;
        used ^= 1;
        if (lane == 0) ptx::bulk_wait_read<DenseCfg::SLABS - 1>();   // the copy that last used this slab has read it
        __syncwarp();
        return s;
    }
    static __device__ __forceinline__ int place(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }
    // units [u0, u0 + 4) of this lane's row
    __device__ __forceinline__ void put4(uint8_t* slab, int u0, const uint32_t* w) const {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(slab + place(lane, u0 + u)) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
    }
    // The slab's rows to rows row.. and columns col.. of `o` (T: its element); M rows exist.
    template <typename T>
    __device__ __forceinline__ void out(uint8_t* slab, const CUtensorMap* map, const DenseOut& o, int row, int col, int z,
                                        int M, long long z_stride) {
        constexpr int PER = 128 / sizeof(T), UNIT = 16 / sizeof(T);
        const int rows = M - row, cols = o.cols - col;   // (a copy rounds a row's end up to 16 bytes)
        if (o.tma && (o.cols % UNIT == 0 || cols >= PER)) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (rows > 0 && cols > 0) ptx::tma_store_3d(map, ptx::smem_u32(slab), col, row, z);
                ptx::bulk_commit();
            }
            return;
        }
        __syncwarp();
        T* c = static_cast<T*>(o.p) + z * z_stride + static_cast<long long>(row) * o.ld + col;
#pragma unroll 4
        for (int r = 0; r < min(rows, 32); ++r) {
#pragma unroll
            for (int i = lane; i < PER; i += 32)
                if (i < cols) c[r * o.ld + i] = reinterpret_cast<const T*>(slab + place(r, i / UNIT))[i % UNIT];
        }
        __syncwarp();
        if (lane == 0) ptx::bulk_commit();   // (an empty group: every slab used counts as one)
    }
};

// e and the sum of 32 logits of a row, relative to 2^ref; columns from `cols` on do not exist.
__device__ __forceinline__ float dense_exps(uint32_t (&r)[32], float ref, int cols) {
    float s0 = 0.0f, s1 = 0.0f;
    if (cols < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i >= cols) r[i] = 0xff800000u;   // minus infinity
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float a = ptx::exp2_approx(fmaf(__uint_as_float(r[i]), 1.4426950408889634f, -ref));
        const float b = ptx::exp2_approx(fmaf(__uint_as_float(r[i + 1]), 1.4426950408889634f, -ref));
        s0 += a;
        s1 += b;
        r[i] = __float_as_uint(a);
        r[i + 1] = __float_as_uint(b);
    }
    return s0 + s1;
}

// Sums of exponentials in this range need no exponent taken out: none of the summands that
// matter is near the ends of bf16's (or fp32's) range.
__device__ __forceinline__ bool dense_plain_sum(float s) { return s > 5.4e-20f && s < 1.8e19f; }

// The power of two to take out of exponentials whose largest logit is `top`: none where that is
// infinite (the exponentials are zeros or infinities then, and stay so).
__device__ __forceinline__ float dense_exponent(float top) {
    return fabsf(top) < __int_as_float(0x7f800000) ? ceilf(top * 1.4426950408889634f) : 0.0f;
}

template <bool A_MN, bool B_MN, DenseEnd E>
__global__ void __launch_bounds__(DenseCfg::THREADS, 1)
    dense_pair_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                      const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                      const __grid_constant__ CUtensorMap tmC0, const __grid_constant__ CUtensorMap tmC1,
                      const __grid_constant__ CUtensorMap tmC2, const DenseParams p) {
    using C = DenseCfg;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = ptx::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    uint8_t* slabs = smem + C::STAGES * C::STAGE_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(slabs + C::EW * C::SLABS * C::SLAB_BYTES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::NBARS);
    volatile uint32_t* abort_flag = tmem_holder + 1;

    const uint32_t full0 = ptx::smem_u32(bars);
    const uint32_t empty0 = full0 + 8 * C::STAGES;
    const uint32_t accf0 = empty0 + 8 * C::STAGES;
    const uint32_t acce0 = accf0 + 16;
    const uint32_t drain_bar = acce0 + 16;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(full0 + 8 * s, 1);    // the leader's producer and both CTAs' bytes
            ptx::mbar_init(empty0 + 8 * s, 1);   // the MMAs' commit
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(accf0 + 8 * b, 1);
            ptx::mbar_init(acce0 + 8 * b, 2 * C::EW);
        }
        ptx::mbar_init(drain_bar, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmA0);
        ptx::prefetch_tensormap(&tmB0);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(tmem_holder), 512);
        ptx::tmem_relinquish_pair();
    }
    __syncwarp();
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    // nothing above touches global memory; the operands may be the previous kernel's results
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const int units = p.tiles_m * p.tiles_n * p.splits;
    const int u0 = blockIdx.x / 2, ustep = gridDim.x / 2;
    const AbortNet net{ptx::smem_u32(const_cast<uint32_t*>(abort_flag)), 2};
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned int code) {
        return wait_warp_pair(bar, parity, abort_flag, net, p.timeout_ns, p.status, code);
    };

    if (warp == 0) {
        // ------------------------------------------------ operand loads
        const uint32_t full_leader0 = ptx::mapa_shared(full0, 0u);
        uint32_t s = 0, ph = 0;
        bool ok = true;
        for (int u = u0; ok && u < units; u += ustep) {
            const DenseUnit U = dense_unit(p, u);
            const int row = U.m0 + static_cast<int>(rank) * 128;
            const int col = E == DenseEnd::GATE ? U.n * 128 : U.n * C::BN + static_cast<int>(rank) * 128;
            for (int kb = U.lo; kb < U.hi; ++kb) {
                if (!wait(empty0 + 8 * s, ph ^ 1u, DEV_TIMEOUT_PRODUCER)) {
                    ok = false;
                    break;
                }
                const bool second = E == DenseEnd::STORE && kb >= p.kb0;
                const int k = (second ? kb - p.kb0 : kb) * C::BK;
                const CUtensorMap* ma = second ? &tmA1 : &tmA0;
                const CUtensorMap* mb = second || (E == DenseEnd::GATE && rank) ? &tmB1 : &tmB0;
                const uint32_t sa = ptx::smem_u32(smem) + s * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                const uint32_t fb = full_leader0 + 8 * s;
                if (rank == 0) ptx::mbar_arrive_expect_tx_elected(full0 + 8 * s, 2 * C::STAGE_BYTES);
                if constexpr (A_MN) {   // boxes of 64 rows of M × 64 of K
                    ptx::tma_load_2d_pair_elected(sa, ma, fb, row, k);
                    ptx::tma_load_2d_pair_elected(sa + 8192, ma, fb, row + 64, k);
                } else {
                    ptx::tma_load_2d_pair_elected(sa, ma, fb, k, row);
                }
                if constexpr (B_MN) {
                    ptx::tma_load_2d_pair_elected(sb, mb, fb, col, k);
                    ptx::tma_load_2d_pair_elected(sb + 8192, mb, fb, col + 64, k);
                } else {
                    ptx::tma_load_2d_pair_elected(sb, mb, fb, k, col);
                }
                if (++s == C::STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) spin_ns(200000);   // copies issued before the abort land within microseconds
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issue (the pair's leader)
        if (rank == 0) {
            constexpr uint32_t IDESC = ptx::make_idesc(1, 1, A_MN, B_MN, C::BM, C::BN);
            // K contiguous: a k-slice of 16 values is 32 bytes further in the row. Rows contiguous:
            // boxes of 64 rows 8192 bytes apart, a k-slice 16 rows of 128 bytes further.
            constexpr uint64_t A_STEP = A_MN ? 128 : 2, B_STEP = B_MN ? 128 : 2, STEP = C::STAGE_BYTES / 16;
            const uint32_t stage0 = ptx::smem_u32(smem);
            const uint64_t adesc0 = ptx::sdesc_sw128(stage0, A_MN ? 8192 : 16, 1024);
            const uint64_t bdesc0 = ptx::sdesc_sw128(stage0 + C::A_BYTES, B_MN ? 8192 : 16, 1024);
            uint32_t s = 0, ph = 0;
            bool ok = true;
            for (int u = u0, j = 0; ok && u < units; u += ustep, ++j) {
                const DenseUnit U = dense_unit(p, u);
                const uint32_t b = j & 1;
                if (!wait(acce0 + 8 * b, ((j >> 1) & 1) ^ 1u, DEV_TIMEOUT_MMA_ACC)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                for (int kb = U.lo; kb < U.hi; ++kb) {
                    if (!wait(full0 + 8 * s, ph, DEV_TIMEOUT_MMA_FULL)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint64_t ad = adesc0 + s * STEP, bd = bdesc0 + s * STEP;
                    ptx::mma_f16_pair_x4_elected(tmem_base + b * C::BN, ad, bd, ad + A_STEP, bd + B_STEP, ad + 2 * A_STEP,
                                                 bd + 2 * B_STEP, ad + 3 * A_STEP, bd + 3 * B_STEP, IDESC,
                                                 kb > U.lo ? 1u : 0u);
                    ptx::mma_commit_pair_multicast_elected(empty0 + 8 * s, 0x3);
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) ptx::mma_commit_pair_multicast_elected(accf0 + 8 * b, 0x3);
            }
            if (!ok) {
                ptx::mma_commit_pair_multicast_elected(drain_bar, 0x1);
                if (lane == 0) wait_drain(drain_bar, 0, p.timeout_ns);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ the ends
        const int quarter = warp & 3;         // the tensor-memory lanes this warp may read
        const int h = (warp - 2) >> 2;        // its share of the columns
        const uint32_t acce_leader0 = ptx::mapa_shared(acce0, 0u);
        DenseSlabs out{slabs + (warp - 2) * C::SLABS * C::SLAB_BYTES, 0, lane};
        for (int u = u0, j = 0; u < units; u += ustep, ++j) {
            const DenseUnit U = dense_unit(p, u);
            const uint32_t b = j & 1;
            const int row0 = U.m0 + static_cast<int>(rank) * 128 + quarter * 32, row = row0 + lane;
            if (!wait(accf0 + 8 * b, (j >> 1) & 1, DEV_TIMEOUT_EPILOGUE)) break;
            ptx::tc_fence_after();
            auto release = [&]() {   // the accumulator is read: free for the tile after the next
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster_relaxed(acce_leader0 + 8 * b);
            };
            const uint32_t t = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + b * C::BN;
            if constexpr (E == DenseEnd::STORE) {
                const uint32_t th = t + h * 128;
                const int col0 = U.n * C::BN + h * 128;
                const float f = p.factor && row < p.M ? p.factor[row] : 1.0f;
                const float* plus = p.plus && row < p.M ? p.plus + static_cast<long long>(row) * p.ld_plus : nullptr;
                const long long z_stride = static_cast<long long>(p.M) * p.out[0].ld;
                auto values = [&](uint32_t (&r)[32], int c) {
                    ptx::tmem_ld_32x32b_x32(th + c, r);
                    ptx::tmem_ld_wait(r);
                    if (c == 96) release();
                    if (p.factor) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            r[i] = f == 0.0f ? 0u : __float_as_uint(__uint_as_float(r[i]) * f);
                    }
                    if (plus) {   // (rows of whole 16-byte pieces, in a workspace)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            if (col0 + c + i >= p.N) continue;
                            const float4 x = *reinterpret_cast<const float4*>(plus + col0 + c + i);
                            r[i] = __float_as_uint(__uint_as_float(r[i]) + x.x);
                            r[i + 1] = __float_as_uint(__uint_as_float(r[i + 1]) + x.y);
                            r[i + 2] = __float_as_uint(__uint_as_float(r[i + 2]) + x.z);
                            r[i + 3] = __float_as_uint(__uint_as_float(r[i + 3]) + x.w);
                        }
                    }
                };
                if (p.f32) {
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t r[32];
                        values(r, c);
                        uint8_t* slab = out.take();
                        out.put4(slab, 0, r);
                        out.put4(slab, 4, r + 16);
                        out.out<float>(slab, &tmC0, p.out[0], row0, col0 + c, U.z, p.M, z_stride);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < 128; c += 64) {
                        uint32_t w[32];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t r[32];
                            values(r, c + 32 * k);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[16 * k + i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                        }
                        uint8_t* slab = out.take();
                        out.put4(slab, 0, w);
                        out.put4(slab, 4, w + 16);
                        out.out<__nv_bfloat16>(slab, &tmC0, p.out[0], row0, col0 + c, U.z, p.M, z_stride);
                    }
                }
            } else if constexpr (E == DenseEnd::GATE) {
                const uint32_t th = t + h * 64;
                const int col0 = U.n * 128 + h * 64;
                uint8_t* slab = out.take();
#pragma unroll 1
                for (int c = 0; c < 64; c += 32) {
                    uint32_t g[32], x[32], w[16];
                    ptx::tmem_ld_32x32b_x32(th + c, g);
                    ptx::tmem_ld_32x32b_x32(th + 128 + c, x);
                    ptx::tmem_ld_wait(g);
                    ptx::tmem_ld_wait(x);
                    float unused;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[i] = pack_bf16(dense_act<false>(p.act, __uint_as_float(g[2 * i]), unused) * __uint_as_float(x[2 * i]),
                                         dense_act<false>(p.act, __uint_as_float(g[2 * i + 1]), unused) *
                                             __uint_as_float(x[2 * i + 1]));
                    out.put4(slab, c / 8, w);
                }
                out.out<__nv_bfloat16>(slab, &tmC0, p.out[0], row0, col0, 0, p.M, 0);
                if (p.out[1].p) {
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        slab = out.take();
#pragma unroll
                        for (int c = 0; c < 64; c += 32) {
                            uint32_t g[32], w[16];
                            ptx::tmem_ld_32x32b_x32(th + 128 * k + c, g);
                            ptx::tmem_ld_wait(g);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = pack_bf16(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]));
                            out.put4(slab, c / 8, w);
                        }
                        out.out<__nv_bfloat16>(slab, k ? &tmC2 : &tmC1, k ? p.out[2] : p.out[1], row0, col0, 0, p.M, 0);
                    }
                }
                release();
            } else if constexpr (E == DenseEnd::GATE_GRAD) {
                const uint32_t th = t + h * 128;
                const int col0 = U.n * C::BN + h * 128;
                const long long at = static_cast<long long>(row) * p.ld_kept;
#pragma unroll 1
                for (int c = 0; c < 128; c += 64) {
                    uint32_t wg[32], wu[32];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int col = col0 + c + 32 * k;
                        uint4 g4[4], u4[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bool in = row < p.M && col + 8 * i < p.N;   // (the buffers' rows are whole pieces)
                            g4[i] = in ? *reinterpret_cast<const uint4*>(p.gate + at + col + 8 * i) : make_uint4(0, 0, 0, 0);
                            u4[i] = in ? *reinterpret_cast<const uint4*>(p.up + at + col + 8 * i) : make_uint4(0, 0, 0, 0);
                        }
                        uint32_t r[32];
                        ptx::tmem_ld_32x32b_x32(th + c + 32 * k, r);
                        ptx::tmem_ld_wait(r);
                        if (c + 32 * k == 96) release();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint32_t g2 = (&g4[i / 4].x)[i % 4], x2 = (&u4[i / 4].x)[i % 4];
                            float dg[2], du[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float g = __uint_as_float(e ? g2 & 0xffff0000u : g2 << 16);
                                const float x = __uint_as_float(e ? x2 & 0xffff0000u : x2 << 16);
                                const float d = __uint_as_float(r[2 * i + e]);
                                float slope;
                                const float a = dense_act<true>(p.act, g, slope);
                                dg[e] = d * x * slope;
                                du[e] = d * a;
                            }
                            wg[16 * k + i] = pack_bf16(dg[0], dg[1]);
                            wu[16 * k + i] = pack_bf16(du[0], du[1]);
                        }
                    }
                    uint8_t* slab = out.take();
                    out.put4(slab, 0, wg);
                    out.put4(slab, 4, wg + 16);
                    out.out<__nv_bfloat16>(slab, &tmC0, p.out[0], row0, col0 + c, 0, p.M, 0);
                    slab = out.take();
                    out.put4(slab, 0, wu);
                    out.put4(slab, 4, wu + 16);
                    out.out<__nv_bfloat16>(slab, &tmC1, p.out[1], row0, col0 + c, 0, p.M, 0);
                }
            } else {
                const uint32_t th = t + h * 128;
                const int col0 = U.n * C::BN + h * 128;
                long long target = -1;
                if (row < p.M)
                    target = p.wide_targets ? static_cast<const long long*>(p.targets)[row]
                                            : static_cast<const int*>(p.targets)[row];
                const bool kept = target >= 0 && target < p.N;
                const int mine = kept ? static_cast<int>(target) - col0 : -1;   // the target's column in this warp's
                uint8_t *slab = nullptr, *slab1 = nullptr;   // the first and the second 64 columns
                float sum = 0.0f, ref = 0.0f;
                // relative to 1; where a row's sum comes out too large or too small for that (or NaN), once more
                // relative to the largest logit's exponential
                auto exps = [&](bool first) {
                    sum = 0.0f;
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t r[32];
                        ptx::tmem_ld_32x32b_x32(th + c, r);
                        ptx::tmem_ld_wait(r);
                        if (first && __any_sync(0xffffffffu, mine >= c && mine < c + 32)) {
                            float v = 0.0f;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (mine == c + i) v = __uint_as_float(r[i]);
                            if (mine >= c && mine < c + 32) p.target_logit[row] = v;
                        }
                        sum += dense_exps(r, ref, p.N - col0 - c);
                        if (p.exps) {
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = kept ? pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])) : 0u;
                            out.put4(c < 64 ? slab : slab1, c % 64 / 8, w);
                        }
                    }
                };
                if (p.exps) {
                    slab = out.take();
                    slab1 = out.base + out.used * C::SLAB_BYTES;
                    if (lane == 0) ptx::bulk_wait_read<0>();
                    __syncwarp();
                    out.used ^= 1;
                }
                exps(true);
                const bool exists = col0 < p.N && row < p.M;
                if (__any_sync(0xffffffffu, exists && !dense_plain_sum(sum))) {
                    float top = __int_as_float(0xff800000);
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t r[32];
                        ptx::tmem_ld_32x32b_x32(th + c, r);
                        ptx::tmem_ld_wait(r);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (col0 + c + i < p.N) top = fmaxf(top, __uint_as_float(r[i]));
                    }
                    if (!dense_plain_sum(sum)) ref = dense_exponent(top);
                    exps(false);
                }
                release();
                if (exists) p.parts[static_cast<long long>(col0 / 128) * p.M + row] = make_float2(ref, sum);
                if (p.exps) {
                    out.out<__nv_bfloat16>(slab, &tmC0, p.out[0], row0, col0, 0, p.M, 0);
                    out.out<__nv_bfloat16>(slab1, &tmC0, p.out[0], row0, col0 + 64, 0, p.M, 0);
                }
            }
            __syncwarp();
        }
        if (lane == 0) ptx::bulk_wait<0>();
        __syncwarp();
    }

    // ------------------------------------------------ teardown
    ptx::tc_fence_before();
    ptx::cluster_sync();   // no CTA frees TMEM or exits while its peer may still signal it
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace tcl
