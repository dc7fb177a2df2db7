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
//              logit, and in training the exponentials themselves in bf16 (k_dense_rows.cu says
//              what they are relative to)
//
// What is rounded to bf16 on the way from one product to the next, and why. The tensor core multiplies bf16 by bf16;
// an fp32 operand would be read as TF32 (half of the rate, twice the bytes) or in two bf16 parts (twice the MMAs).
// Errors by norm against 64 bits; the last rounding of a bf16 result alone makes 1.65e-3 of it.
//   h                     the down product's operand: out 2.3e-3
//   gate, up              kept for the gradients: 4 bytes a token and inner column, fp32 8. The block's gradients are
//                         off by 2.9e-3 to 3.1e-3; with fp32 copies 2.4e-3
//   dgate, dup            operands of three products
//   the exponentials      operands of both of the entropy's gradients, 2 bytes a token and word; the sums that divide
//                         them are of the unrounded ones (dx 2.2e-3)
//   x·grad/S              the rows of x for dW: the tokens are what that product sums over, so their factors cannot
//                         wait for its end; they go into the smaller operand (dW 2.7e-3)
// Sums are the tensor core's fp32 ones, which are cut off, not rounded: by 2^-23 of a partial sum at most for each 16
// terms, 5e-6 of the result in all where 4096 of them have one sign (k_dense_rows.cu says what becomes of that in a loss).
//
// Roles of each CTA: warp 0 loads A, warp 10 B (TMA, 128-byte swizzle, a ring of 64-value k-blocks),
// warp 1 of the pair's leader issues the MMAs into one of two accumulators in tensor memory, warps 2
// to 9 read the other one (each 32 lanes × half of the columns, or four of them all columns) and store through
// slabs of 32 rows × 128 bytes, copied out by the tensor copy engine. A pair walks its tiles blockIdx/2, + pairs, ...
//
// Every wait is bounded; a role that gives up raises the pair's abort flag.
#pragma once

#include <type_traits>

#include "gemm_kernel_pair.cuh"
#include "rows8.cuh"

namespace tcl {

enum class DenseEnd : int { STORE, GATE, GATE_GRAD, ENTROPY };
enum : int { DENSE_SILU = 0, DENSE_GELU = 1, DENSE_GELU_TANH = 2 };
constexpr int kDenseProblems = 4;   // of one launch

struct DenseOut {
    void* p;
    long long ld;     // elements
    int cols;         // columns that may be written (a buffer of this library's own: whole 16-byte pieces)
    int tma;          // rows start on 16-byte pieces: there is a tensor map
};

// One D = A·B^T of a launch.
struct DenseProblem {
    int M, N;              // rows and columns of D (GATE: N columns of h)
    int kb0, kb1;          // k-blocks of the first and of the second operand pair (0: one pair)
    int tiles_m, tiles_n, splits;
    int first;             // its first unit
    int a_mn, b_mn;        // STORE: rows (not K) contiguous; the other ends: both K, GATE_GRAD B's rows
    int a_3d, b_3d;        // rows contiguous: both boxes of 64 rows in one copy (3-D maps of whole chunks of 64 rows)
    int f32;               // STORE: fp32 result
    DenseOut out;          // D, h or dgate or the exponentials
    const float* factor;   // STORE: of each row (NULL: ones); a row whose factor is zero is zeros
    const float* plus;     // STORE: added to the result (NULL: nothing); rows of whole 16-byte pieces
    long long ld_plus;
};

struct DenseMaps {
    // (STORE: for each problem; the other ends: c for each result, GATE_GRAD a[1] gate and up)
    CUtensorMap a[kDenseProblems][2], b[kDenseProblems][2], c[kDenseProblems];
};

struct DenseParams {
    DenseProblem q[kDenseProblems];
    int n, units;
    // How units are dealt out to the pairs of SMs: the first long_units of them (of one problem, those with the
    // longest K ranges) in turn; `extra` units of the rest to each pair that got one fewer; then
    // the others in turn. Everyone ends within about one unit of the others.
    int long_units, extra;
    int deep;              // STORE, GATE, wide tiles: a ring of six k-blocks and one staging slab a warp (else five and two);
                           // ENTROPY, wide tiles that store nothing: 2, a ring of seven; GATE_GRAD, wide tiles: a ring of six,
                           // the tile's end by four warps (else five and eight)
    int act;
    DenseOut more[2];      // GATE: gate, up (no address: not asked for); GATE_GRAD: dup
    const void* targets;   // ENTROPY: M of them, int32 or int64
    int wide_targets;
    float2* parts;         // ENTROPY: [chunk of BN/2 columns][row of D]: exponent taken out, sum
    float* target_logit;   // ENTROPY: [row of D]
    int exps;              // ENTROPY: store the exponentials
    unsigned long long timeout_ns;
    unsigned int* status;
};

// Phi(-a) for a >= 0, with ex = exp(-a^2/2): ex·t·P(t), t = 1/(1 + 0.33 a), P fitted to
// exp(a^2/2)·Phi(-a)/t over all a >= 0 (least largest relative error: 1e-6).
__device__ __forceinline__ float dense_normal_tail(float a, float ex) {
    const float t = __fdividef(1.0f, fmaf(0.33f, a, 1.0f));
    float v = 0.033285726f;
    v = fmaf(v, t, -0.10566493f);
    v = fmaf(v, t, 0.067431189f);
    v = fmaf(v, t, 0.033428829f);
    v = fmaf(v, t, 0.091004848f);
    v = fmaf(v, t, 0.11721677f);
    v = fmaf(v, t, 0.13164698f);
    v = fmaf(v, t, 0.13165107f);
    return ex * t * v;
}

// act(g), and its derivative where it is asked for.
template <int ACT, bool SLOPE>
__device__ __forceinline__ float dense_act(float g, float& slope) {
    if constexpr (ACT == DENSE_GELU) {
        const float ex = ptx::exp2_approx(-0.72134752044448170f * g * g);
        const float q = dense_normal_tail(fabsf(g), ex), p = g > 0.0f ? 1.0f - q : q;
        if (SLOPE) slope = fmaf(g * 0.39894228040143268f, ex, p);
        return g * p;
    } else {
        float z = -1.4426950408889634f * g;
        if constexpr (ACT == DENSE_GELU_TANH) z *= 1.5957691216057308f * fmaf(0.044715f * g, g, 1.0f);   // (1 + tanh(y))/2 = 1/(1 + exp(-2y))
        const float s = __fdividef(1.0f, 1.0f + ptx::exp2_approx(z));
        if constexpr (SLOPE && ACT == DENSE_GELU_TANH) {
            const float c = fminf(fmaxf(g, -1e4f), 1e4f);   // (s(1 - s) is zero long before that)
            slope = fmaf(c * s * (1.0f - s), 1.5957691216057308f * fmaf(0.134145f * c, c, 1.0f), s);
        } else if constexpr (SLOPE) {
            slope = s * fmaf(g, 1.0f - s, 1.0f);
        }
        return g * s;
    }
}

// f with the activation as a compile-time number: the loops over a tile's values must stay short, since
// what does not fit the instruction cache is fetched again by every warp (all three activations
// in one unrolled loop of 64 values: 35 us a tile instead of 5).
template <class F>
__device__ __forceinline__ void dense_with_act(int act, F f) {
    if (act == DENSE_SILU)
        f(std::integral_constant<int, DENSE_SILU>());
    else if (act == DENSE_GELU)
        f(std::integral_constant<int, DENSE_GELU>());
    else
        f(std::integral_constant<int, DENSE_GELU_TANH>());
}

template <int BN_>
struct DenseCfg {
    static constexpr int BM = 256, BN = BN_, BK = 64;
    static constexpr int CW = BN / 2;               // columns of an epilogue warp
    // Wide tiles have room for five k-blocks and two staging slabs a warp, or for six and one: the sixth where K is
    // long (hidden 4096, inner 14336, gate and up kept: 512 tokens 123 us to 118, 2048 tokens 411 to 400;
    // gradients of 300 tokens 213 to 201, of 1023 tokens 413 to 405), the second slab where k-blocks are few and the
    // ends show (gradients of 100 tokens 153 us, 169 with one slab).
    static constexpr int STAGES = BN == 256 ? 5 : 6;
    static constexpr int MOST_STAGES = 7;
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BN / 2 * 128;   // a CTA's share of a k-block
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EW = 8;                    // epilogue warps
    static constexpr int SLABS = 2, SLAB_BYTES = 32 * 128;
    static constexpr int NBARS = 2 * MOST_STAGES + 5 + EW;   // (a warp's own: GATE_GRAD)
    static constexpr int B_WARP = 2 + EW;           // the warp that loads B
    static constexpr int THREADS = 96 + 32 * EW;
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EW * SLABS * SLAB_BYTES + (NBARS + 2) * 8;
    static_assert(BN != 256 || STAGE_BYTES == EW * SLAB_BYTES, "a k-block for a slab of each warp");
    static_assert(SMEM_BYTES <= 232448, "exceeds the 227 KB per-block shared memory limit");
};

struct DenseUnit {
    int q, m0, n, z, lo, hi;   // problem, first row, tile column, K range's number and k-blocks
};

// The unit at step j of pair r of `pairs`; p.units or more: none is left.
__device__ __forceinline__ int dense_walk(const DenseParams& p, int r, int pairs, int j) {
    const int r0 = p.long_units % pairs, mine = p.long_units / pairs + (r < r0 ? 1 : 0);
    if (j < mine) return j * pairs + r;
    j -= mine;
    if (r < r0) return p.long_units + p.extra * (pairs - r0) + j * pairs + r;
    if (j < p.extra) return p.long_units + j * (pairs - r0) + r - r0;
    return p.long_units + p.extra * (pairs - r0) + (j - p.extra) * pairs + r;
}

template <DenseEnd E>
__device__ __forceinline__ DenseUnit dense_unit(const DenseParams& p, int u) {
    // eight tile rows share a pass over the tile columns, so that a wave of the GPU reads few
    // operand rows of either side
    constexpr int G = 8;
    DenseUnit U;
    U.q = 0;
    if constexpr (E == DenseEnd::STORE)
        while (U.q + 1 < p.n && u >= p.q[U.q + 1].first) ++U.q;
    const DenseProblem& q = p.q[U.q];
    u -= q.first;
    const int tiles = q.tiles_m * q.tiles_n, z = u / tiles, t = u - z * tiles;
    const int g = t / (G * q.tiles_n) * G, gn = min(G, q.tiles_m - g), r = t - g * q.tiles_n;
    const long long kb = q.kb0 + q.kb1;
    U.m0 = (g + r % gn) * 256;
    U.n = r / gn;
    U.z = z;
    U.lo = static_cast<int>(kb * z / q.splits);
    U.hi = static_cast<int>(kb * (z + 1) / q.splits);
    return U;
}

// A warp's staging slabs, taken in turn: 32 rows (a lane each) of 128 bytes, 16-byte units
// permuted by the row as the tensor copies do.
struct DenseSlabs {
    uint8_t* base;
    int used, lane;
    bool one;
    __device__ __forceinline__ uint8_t* take() {
        uint8_t* s = base + used * DenseCfg<256>::SLAB_BYTES;
        if (!one) used ^= 1;
        if (lane == 0) {   // the copy that last used this slab has read it
            if (one)
                ptx::bulk_wait_read<0>();
            else
                ptx::bulk_wait_read<1>();
        }
        __syncwarp();
        return s;
    }
    // The other slab too, right after take().
    __device__ __forceinline__ uint8_t* take_other() {
        uint8_t* s = base + used * DenseCfg<256>::SLAB_BYTES;
        used ^= 1;
        if (lane == 0) ptx::bulk_wait_read<0>();
        __syncwarp();
        return s;
    }
    static __device__ __forceinline__ int place(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }
    // N units of this lane's row from u0 on
    template <int N>
    __device__ __forceinline__ void put(uint8_t* slab, int u0, const uint32_t* w) const {
#pragma unroll
        for (int u = 0; u < N; ++u)
            *reinterpret_cast<uint4*>(slab + place(lane, u0 + u)) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
    }
    template <int N>
    __device__ __forceinline__ void get(const uint8_t* slab, int u0, uint32_t* w) const {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint4 v = *reinterpret_cast<const uint4*>(slab + place(lane, u0 + u));
            w[4 * u] = v.x;
            w[4 * u + 1] = v.y;
            w[4 * u + 2] = v.z;
            w[4 * u + 3] = v.w;
        }
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
        // a 32-bit word a lane, two elements of bf16 rows that start on words; eight rows are read before the first
        // of them is stored (a load waits for no store then: a slab takes 1,100 cycles instead of 4,400)
        const bool words = sizeof(T) == 4 || (o.ld % 2 == 0 && reinterpret_cast<uintptr_t>(o.p) % 4 == 0);
        constexpr int E = 4 / sizeof(T);   // elements of a word
#pragma unroll 1
        for (int r0 = 0; r0 < min(rows, 32); r0 += 8) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const uint32_t*>(slab + place(r0 + i, lane / 4) + lane % 4 * 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                T* to = c + (r0 + i) * o.ld + lane * E;
                if (r0 + i >= rows) continue;
                if (words && lane * E + E <= cols) {
                    *reinterpret_cast<uint32_t*>(to) = v[i];
                } else if constexpr (E == 2) {
                    if (2 * lane < cols) reinterpret_cast<uint16_t*>(to)[0] = static_cast<uint16_t>(v[i]);
                    if (2 * lane + 1 < cols) reinterpret_cast<uint16_t*>(to)[1] = static_cast<uint16_t>(v[i] >> 16);
                }
            }
        }
        __syncwarp();
        if (lane == 0) ptx::bulk_commit();   // (an empty group: every slab used counts as one)
    }
};

// The exponentials of 32 logits of a row, relative to 2^ref, and their sum; columns from `cols` on do not exist.
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

// The power of two to take out of exponentials whose largest logit is `top`: none where that is beyond 2^30,
// infinities among them (the exponentials are zeros or infinities then, and stay so). There fp32's numbers are 128
// apart, and the product with log2(e), rounded, misses the exponent by so much that the exponentials would come
// out as either all the same: a large logit as if it were not there. Up to 2^30 it misses it by 64 at most, which the
// sums have room for.
__device__ __forceinline__ float dense_exponent(float top) {
    return fabsf(top) <= 0x1p30f ? ceilf(top * 1.4426950408889634f) : 0.0f;
}

// Adds a chunk's sum, relative to 2^ref, to a row's.
__device__ __forceinline__ void dense_merge(float& to_ref, float& to_sum, float ref, float sum) {
    constexpr float INF = __builtin_huge_valf();
    if (sum == 0.0f) return;
    if (to_sum == 0.0f) {
        to_ref = ref;
        to_sum = sum;
    } else if (sum == INF || to_sum == INF) {   // (of an infinite logit: times a power of two that is zero it would be NaN)
        to_sum += sum;
    } else if (ref <= to_ref) {
        to_sum += ref == to_ref ? sum : sum * exp2f(ref - to_ref);
    } else {
        to_sum = to_sum * exp2f(to_ref - ref) + sum;
        to_ref = ref;
    }
}

template <int BN, DenseEnd E>
__global__ void __launch_bounds__(DenseCfg<BN>::THREADS, 1)
    dense_pair_kernel(const __grid_constant__ DenseMaps maps, const __grid_constant__ DenseParams p) {
    using C = DenseCfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = ptx::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    const bool deep = BN == 256 && E != DenseEnd::ENTROPY && p.deep;
    const uint32_t stages = C::STAGES + (BN == 256 ? p.deep : 0);
    uint8_t* slabs = smem + stages * C::STAGE_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE_BYTES + C::EW * C::SLABS * C::SLAB_BYTES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::NBARS);
    volatile uint32_t* abort_flag = tmem_holder + 1;

    const uint32_t full0 = ptx::smem_u32(bars);
    const uint32_t empty0 = full0 + 8 * C::MOST_STAGES;
    const uint32_t accf0 = empty0 + 8 * C::MOST_STAGES;
    const uint32_t acce0 = accf0 + 16;
    const uint32_t drain_bar = acce0 + 16;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::MOST_STAGES; ++s) {
            ptx::mbar_init(full0 + 8 * s, 1);    // the leader's producer and both CTAs' bytes
            ptx::mbar_init(empty0 + 8 * s, 1);   // the MMAs' commit
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(accf0 + 8 * b, 1);
            ptx::mbar_init(acce0 + 8 * b, 2 * C::EW);
        }
        ptx::mbar_init(drain_bar, 1);
        for (int w = 0; w < C::EW; ++w) ptx::mbar_init(drain_bar + 8 + 8 * w, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&maps.a[0][0]);
        ptx::prefetch_tensormap(&maps.b[0][0]);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(tmem_holder), C::TMEM_COLS);
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

    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const AbortNet net{ptx::smem_u32(const_cast<uint32_t*>(abort_flag)), 2};
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned int code) {
        return wait_warp_pair(bar, parity, abort_flag, net, p.timeout_ns, p.status, code);
    };

    if (warp == 0 || warp == C::B_WARP) {
        // ------------------------------------------------ operand loads: a warp for A, one for B
        // (What a warp does for a k-block, waiting for its slot and issuing a copy or two, takes it some 400 cycles
        // for both operands: with one warp, tiles whose operands both have contiguous rows took 640 cycles a
        // k-block, 512 of them the MMAs'.)
        const bool of_a = warp == 0;
        const uint32_t full_leader0 = ptx::mapa_shared(full0, 0u);
        const uint32_t to0 = ptx::smem_u32(smem) + (of_a ? 0 : C::A_BYTES);
        uint32_t s = 0, ph = 0;
        bool ok = true;
        for (int j = 0, u; ok && (u = dense_walk(p, pair, pairs, j)) < p.units; ++j) {
            const DenseUnit U = dense_unit<E>(p, u);
            const DenseProblem& q = p.q[U.q];
            const bool mn = of_a ? E == DenseEnd::STORE && q.a_mn
                                 : E == DenseEnd::GATE_GRAD || (E == DenseEnd::STORE && q.b_mn);
            const bool whole = of_a ? q.a_3d : q.b_3d, two = of_a || BN == 256;   // (boxes of 64 rows)
            const int at = of_a ? U.m0 + static_cast<int>(rank) * 128
                                : E == DenseEnd::GATE ? U.n * C::CW : U.n * BN + static_cast<int>(rank) * C::CW;
            const CUtensorMap* map0 = of_a ? &maps.a[U.q][0] : &maps.b[U.q][E == DenseEnd::GATE ? static_cast<int>(rank) : 0];
            const CUtensorMap* map1 = of_a ? &maps.a[U.q][1] : &maps.b[U.q][1];
            const int kb0 = E == DenseEnd::STORE ? q.kb0 : U.hi;   // the k-block from which on the second pair counts
            // a run of k-blocks through one of the loops below; `load` issues a k-block's copies
            auto run = [&](auto load) {
                for (int kb = U.lo; kb < U.hi; ++kb) {
                    if (!wait(empty0 + 8 * s, ph ^ 1u, DEV_TIMEOUT_PRODUCER)) return false;
                    const bool second = kb >= kb0;
                    if (of_a && rank == 0) ptx::mbar_arrive_expect_tx_elected(full0 + 8 * s, 2 * C::STAGE_BYTES);
                    load(to0 + s * C::STAGE_BYTES, second ? map1 : map0, full_leader0 + 8 * s, (second ? kb - kb0 : kb) * C::BK);
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                return true;
            };
            if (!mn)
                ok = run([&](uint32_t to, const CUtensorMap* m, uint32_t bar, int k) { ptx::tma_load_2d_pair_elected(to, m, bar, k, at); });
            else if (whole)
                ok = run([&](uint32_t to, const CUtensorMap* m, uint32_t bar, int k) {
                    ptx::tma_load_3d_pair_elected(to, m, bar, 0, k, at / 64);
                });
            else
                ok = run([&](uint32_t to, const CUtensorMap* m, uint32_t bar, int k) {
                    ptx::tma_load_2d_pair_elected(to, m, bar, at, k);
                    if (two) ptx::tma_load_2d_pair_elected(to + 8192, m, bar, at + 64, k);
                });
        }
        if (!ok && lane == 0) spin_ns(200000);   // copies issued before the abort land within microseconds
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issue (the pair's leader)
        if (rank == 0) {
            constexpr uint64_t STEP = C::STAGE_BYTES / 16;
            const uint32_t stage0 = ptx::smem_u32(smem);
            uint32_t s = 0, ph = 0;
            bool ok = true;
            for (int j = 0, u; ok && (u = dense_walk(p, pair, pairs, j)) < p.units; ++j) {
                const DenseUnit U = dense_unit<E>(p, u);
                const DenseProblem& q = p.q[U.q];
                const bool a_mn = E == DenseEnd::STORE && q.a_mn;
                const bool b_mn = E == DenseEnd::GATE_GRAD || (E == DenseEnd::STORE && q.b_mn);
                const uint32_t idesc = ptx::make_idesc(1, 1, a_mn, b_mn, C::BM, BN);
                // K contiguous: a k-slice of 16 values is 32 bytes further in the row. Rows contiguous:
                // boxes of 64 rows 8192 bytes apart, a k-slice 16 rows of 128 bytes further.
                const uint64_t as = a_mn ? 128 : 2, bs = b_mn ? 128 : 2;
                const uint64_t adesc0 = ptx::sdesc_sw128(stage0, a_mn ? 8192 : 16, 1024);
                const uint64_t bdesc0 = ptx::sdesc_sw128(stage0 + C::A_BYTES, b_mn ? 8192 : 16, 1024);
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
                    ptx::mma_f16_pair_x4_elected(tmem_base + b * BN, ad, bd, ad + as, bd + bs, ad + 2 * as, bd + 2 * bs,
                                                 ad + 3 * as, bd + 3 * bs, idesc, kb > U.lo ? 1u : 0u);
                    ptx::mma_commit_pair_multicast_elected(empty0 + 8 * s, 0x3);
                    if (++s == stages) {
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
        DenseSlabs out{slabs + (warp - 2) * (deep && E != DenseEnd::GATE_GRAD ? 1 : C::SLABS) * C::SLAB_BYTES, 0, lane, deep};
        [[maybe_unused]] uint32_t kept_phase = 0;
        for (int j = 0, u; (u = dense_walk(p, pair, pairs, j)) < p.units; ++j) {
            const DenseUnit U = dense_unit<E>(p, u);
            const DenseProblem& q = p.q[U.q];
            const uint32_t b = j & 1;
            const int row0 = U.m0 + static_cast<int>(rank) * 128 + quarter * 32, row = row0 + lane;
            const int col0 = U.n * BN + h * C::CW;                            // (GATE: of the two tiles side by side)
            const uint32_t t = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + b * BN;
            const uint32_t th = t + h * C::CW;
            auto release = [&]() {   // the accumulator is read: free for the tile after the next
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster_relaxed(acce_leader0 + 8 * b);
            };
            if constexpr (E == DenseEnd::STORE) {
                const float f = q.factor && row < q.M ? q.factor[row] : 1.0f;
                if (!wait(accf0 + 8 * b, (j >> 1) & 1, DEV_TIMEOUT_EPILOGUE)) break;
                ptx::tc_fence_after();
                const float* plus = q.plus && row < q.M ? q.plus + static_cast<long long>(row) * q.ld_plus : nullptr;
                const long long z_stride = static_cast<long long>(q.M) * q.out.ld;
                auto values = [&](uint32_t (&r)[32], int c) {
                    ptx::tmem_ld_32x32b_x32(th + c, r);
                    ptx::tmem_ld_wait(r);
                    if (c + 32 == C::CW) release();
                    if (q.factor) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            r[i] = f == 0.0f ? 0u : __float_as_uint(__uint_as_float(r[i]) * f);
                    }
                    if (plus) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            if (col0 + c + i >= q.N) continue;
                            const float4 x = *reinterpret_cast<const float4*>(plus + col0 + c + i);
                            r[i] = __float_as_uint(__uint_as_float(r[i]) + x.x);
                            r[i + 1] = __float_as_uint(__uint_as_float(r[i + 1]) + x.y);
                            r[i + 2] = __float_as_uint(__uint_as_float(r[i + 2]) + x.z);
                            r[i + 3] = __float_as_uint(__uint_as_float(r[i + 3]) + x.w);
                        }
                    }
                };
                if (q.f32) {
#pragma unroll 1
                    for (int c = 0; c < C::CW; c += 32) {
                        uint32_t r[32];
                        values(r, c);
                        uint8_t* slab = out.take();
                        out.put<8>(slab, 0, r);
                        out.out<float>(slab, &maps.c[U.q], q.out, row0, col0 + c, U.z, q.M, z_stride);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < C::CW; c += 64) {
                        uint8_t* slab = out.take();
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t r[32];
                            values(r, c + 32 * k);
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                            out.put<4>(slab, 4 * k, w);
                        }
                        out.out<__nv_bfloat16>(slab, &maps.c[U.q], q.out, row0, col0 + c, U.z, q.M, z_stride);
                    }
                }
            } else if constexpr (E == DenseEnd::GATE) {
                // half of the tile's CW columns of h to a warp; in a narrow tile the warps of the second
                // half have nothing to do (a slab is 64 columns wide)
                constexpr int W = 64;
                if (!wait(accf0 + 8 * b, (j >> 1) & 1, DEV_TIMEOUT_EPILOGUE)) break;
                ptx::tc_fence_after();
                if (BN == 256 || h == 0) {
                    const uint32_t tg = t + h * W;
                    const int hc = U.n * C::CW + h * W;
                    uint8_t* slab = out.take();
                    dense_with_act(p.act, [&](auto a) {
#pragma unroll 1
                        for (int c = 0; c < W; c += 16) {
                            uint32_t g[16], x[16], w[8];
                            ptx::tmem_ld_32x32b_x16(tg + c, g);
                            ptx::tmem_ld_32x32b_x16(tg + C::CW + c, x);
                            ptx::tmem_ld_wait(g);
                            ptx::tmem_ld_wait(x);
                            float unused;
#pragma unroll
                            for (int i = 0; i < 8; ++i)   // (h's one rounding)
                                w[i] = pack_bf16(
                                    dense_act<decltype(a)::value, false>(__uint_as_float(g[2 * i]), unused) *
                                        __uint_as_float(x[2 * i]),
                                    dense_act<decltype(a)::value, false>(__uint_as_float(g[2 * i + 1]), unused) *
                                        __uint_as_float(x[2 * i + 1]));
                            out.put<2>(slab, c / 8, w);
                        }
                    });
                    out.out<__nv_bfloat16>(slab, &maps.c[0], q.out, row0, hc, 0, q.M, 0);
                    if (p.more[0].p) {
#pragma unroll 1
                        for (int k = 0; k < 2; ++k) {
                            slab = out.take();
#pragma unroll
                            for (int c = 0; c < W; c += 32) {
                                uint32_t g[32], w[16];
                                ptx::tmem_ld_32x32b_x32(tg + C::CW * k + c, g);
                                ptx::tmem_ld_wait(g);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    w[i] = pack_bf16(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]));
                                out.put<4>(slab, c / 8, w);
                            }
                            out.out<__nv_bfloat16>(slab, &maps.c[1 + k], p.more[k], row0, hc, 0, q.M, 0);
                        }
                    }
                }
                release();
            } else if constexpr (E == DenseEnd::GATE_GRAD) {
                // What was kept of 64 columns comes into the two slabs (gate, up) and is replaced there by dgate and
                // dup: a lane reads and writes its own row. The first 64 columns of a tile are fetched before
                // its accumulator is complete, so that they arrive meanwhile.
                uint8_t *sg = out.base, *su = out.base + C::SLAB_BYTES;
                const uint32_t bar = drain_bar + 8 + 8 * (warp - 2);
                auto fetch = [&](int col) {
                    if (lane == 0) {
                        ptx::bulk_wait_read<0>();   // the slabs' last results are copied out
                        ptx::mbar_arrive_expect_tx(bar, 2 * C::SLAB_BYTES);
                        ptx::tma_load_2d(ptx::smem_u32(sg), &maps.a[1][0], bar, col, row0);
                        ptx::tma_load_2d(ptx::smem_u32(su), &maps.a[1][1], bar, col, row0);
                    }
                    __syncwarp();
                };
                const bool mine = !deep || h == 0;   // (a ring of six: half of the warps, all columns each)
                const int cw = deep ? BN : C::CW;
                if (mine) fetch(col0);
                const bool ready = wait(accf0 + 8 * b, (j >> 1) & 1, DEV_TIMEOUT_EPILOGUE);
                ptx::tc_fence_after();
                bool here = true;
                if (!mine)
                    release();
                else dense_with_act(p.act, [&](auto act) {
#pragma unroll 1
                    for (int c = 0; c < cw; c += 64) {
                        if (c) fetch(col0 + c);
                        here = here && wait(bar, kept_phase, DEV_TIMEOUT_EPILOGUE);
                        kept_phase ^= 1u;
                        if (!here || !ready) break;
#pragma unroll 1
                        for (int k = 0; k < 64; k += 16) {
                            uint32_t r[16], wg[8], wu[8];
                            ptx::tmem_ld_32x32b_x16(th + c + k, r);
                            out.get<2>(sg, k / 8, wg);
                            out.get<2>(su, k / 8, wu);
                            ptx::tmem_ld_wait(r);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float dg[2], du[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float g = __uint_as_float(e ? wg[i] & 0xffff0000u : wg[i] << 16);
                                    const float x = __uint_as_float(e ? wu[i] & 0xffff0000u : wu[i] << 16);
                                    const float d = __uint_as_float(r[2 * i + e]);
                                    float slope;
                                    const float a = dense_act<decltype(act)::value, true>(g, slope);
                                    dg[e] = d * x * slope;
                                    du[e] = d * a;
                                }
                                wg[i] = pack_bf16(dg[0], dg[1]);
                                wu[i] = pack_bf16(du[0], du[1]);
                            }
                            out.put<2>(sg, k / 8, wg);
                            out.put<2>(su, k / 8, wu);
                        }
                        if (c + 64 == cw) release();
                        out.out<__nv_bfloat16>(sg, &maps.c[0], q.out, row0, col0 + c, 0, q.M, 0);
                        out.out<__nv_bfloat16>(su, &maps.c[1], p.more[0], row0, col0 + c, 0, q.M, 0);
                    }
                });
                if (!here || !ready) {
                    if (lane == 0) spin_ns(200000);   // copies issued before the abort land within microseconds
                    __syncwarp();
                    break;
                }
            } else {
                long long target = -1;
                if (row < q.M)
                    target = p.wide_targets ? static_cast<const long long*>(p.targets)[row]
                                            : static_cast<const int*>(p.targets)[row];
                if (!wait(accf0 + 8 * b, (j >> 1) & 1, DEV_TIMEOUT_EPILOGUE)) break;
                ptx::tc_fence_after();
                const bool kept = target >= 0 && target < q.N;
                const int mine = kept ? static_cast<int>(target) - col0 : -1;   // the target's column in this warp's
                uint8_t *slab = nullptr, *slab1 = nullptr;   // the first and the second 64 columns
                float sum = 0.0f, ref = 0.0f;
                // relative to 1; where a row's sum comes out too large or too small for that (or NaN), once more
                // relative to the largest logit's exponential
                auto exps = [&](bool first) {
                    sum = 0.0f;
#pragma unroll 1
                    for (int c = 0; c < C::CW; c += 32) {
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
                        sum += dense_exps(r, ref, q.N - col0 - c);
                        if (p.exps) {
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = kept ? pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])) : 0u;
                            out.put<4>(c < 64 ? slab : slab1, c % 64 / 8, w);
                        }
                    }
                };
                if (p.exps) {
                    slab = out.take();
                    if constexpr (BN == 256) slab1 = out.take_other();
                }
                exps(true);
                const bool exists = col0 < q.N && row < q.M;
                if (__any_sync(0xffffffffu, exists && !dense_plain_sum(sum))) {
                    float top = __int_as_float(0xff800000);
#pragma unroll 1
                    for (int c = 0; c < C::CW; c += 32) {
                        uint32_t r[32];
                        ptx::tmem_ld_32x32b_x32(th + c, r);
                        ptx::tmem_ld_wait(r);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (col0 + c + i < q.N) top = fmaxf(top, __uint_as_float(r[i]));
                    }
                    if (!dense_plain_sum(sum)) ref = dense_exponent(top);
                    exps(false);
                }
                release();
                if (exists) p.parts[static_cast<long long>(col0 / C::CW) * q.M + row] = make_float2(ref, sum);
                if (p.exps) {
                    out.out<__nv_bfloat16>(slab, &maps.c[0], q.out, row0, col0, 0, q.M, 0);
                    if constexpr (BN == 256) out.out<__nv_bfloat16>(slab1, &maps.c[0], q.out, row0, col0 + 64, 0, q.M, 0);
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
        ptx::tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace tcl
