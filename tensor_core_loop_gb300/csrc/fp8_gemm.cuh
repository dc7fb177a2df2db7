// Products of e4m3 matrices that carry one fp32 scale for each 128 values of K.
//
// With P_kb the plain product of the operands' k-block kb (128 values of K, or what
// is left of K in the last block),
//   out[p][q] = sum over kb of (sp[p][kb] · sq[q][kb]) · P_kb[p][q]
// where a side's scales belong to its rows or to blocks of 128 rows. A product of two
// e4m3 values is exact in fp32 and the tensor core adds a block's 128 of them in fp32;
// the scales differ from block to block, so each P_kb is taken out of tensor memory and
// added into fp32 registers by one fused multiply-add per element ("promotion"). Past the
// end of K the tensor copies fill in zeros, byte by byte, so K is free.
//
// Roles of a CTA (or of each CTA of a pair of SMs):
//   warp 0      TMA loads of both operands into a ring of 128-byte k-blocks
//   warp 1      issues the MMAs, four per k-block, into a ring of accumulators
//   warps 2, 3  copy each k-block's scales of P and of Q into a ring of shared-memory slots
//               (cp.async: 4-byte pieces, so that scales may have any strides). One warp for
//               both, working out addresses for every k-block, paced the whole kernel.
//   warps 4..   promotion, and the stores of the finished tile
//
// What bounds it: with many rows the promotion, which has to fit beside a k-block's MMAs (512
// cycles of a 256 × 256 tile: per SM quarter 256 cycles of multiply-adds and as many of
// tensor-memory loads); 8192 × 8192 × 4096 takes 200 us, 2.75 PFLOP/s, the tensor pipe busy
// 57 % of the time (without promotion 158 us). Eight warps of 128 sums a thread, two to a
// scheduler, are as many as the registers hold; a few words spilled in the loop cost 30 %.
// With few rows a weight byte's way from HBM bounds it: 16 tokens on 64 experts of 4096 × 2048
// read 319 MB in 51 us, 6.2 TB/s. Scales per column (weight gradients) take two fp32
// operations an element instead of one. There a tile has few k-blocks (32 experts of 2048 × 1024 from
// 32,700 rows: eight, 109 us; 8192 × 4096 × 1000 57 us) and its loads, MMAs, promotion and stores follow
// one another more than they overlap: tensor pipe 26 %, issue slots 41 %, DRAM 35 % busy.
//
// The side in the 128 tensor-memory lanes is P, the one in the columns is Q. Many rows
// of tokens go to P with the weights' rows in Q; few (SWAP) go to Q, as narrow as the
// MMA's N allows, with 128 weight rows in P, so that a weight byte is read once for
// all tokens and no MMA or shared memory is spent on rows that do not exist.
//
// Where one-SM tiles leave most SMs without one, the CTAs of a cluster share a tile's k-blocks
// and one after another's sums are added over distributed shared memory.
//
// Work units are output tiles. Rows sorted by expert come with the experts' offsets on
// the device: every CTA turns them into a running count of tiles, and walks the tiles
// blockIdx, blockIdx + grid, ...; tiles past an expert's end read the next expert's rows
// (harmless: their results are not stored). Rows behind the last expert are written as
// zeros. In weight-gradient form each expert's k-blocks are its own rows, from an offset
// that is a multiple of 128, and experts without rows get zeros.
#pragma once

#include "gemm_kernel_pair.cuh"
#include "rows8.cuh"

namespace tcl {

enum : unsigned int {
    DEV_BAD_OFFSETS = 7,   // expert offsets not ascending from 0 within the rows (or, for weight gradients, off 128)
};

constexpr int kMaxExperts = 1024;
constexpr int kMaxSorted = 256;   // experts that every CTA can put in order in a microsecond

struct Fp8Side {
    const float* scale;
    long long s_row, s_group, s_expert;   // strides in elements
    int block;                            // 1: one scale row for each 128 rows
};

struct Fp8Params {
    Fp8Side P, Q;
    const int* offsets;      // experts + 1 row offsets (NULL: one expert with all rows)
    int experts;
    int rows;                // rows of the token side (weight gradient: values of K)
    int wrows;               // rows of the weight side (weight gradient: rows of P)
    int qrows;               // weight gradient: rows of Q
    int num_kb;              // k-blocks of a tile (weight gradient: given by the offsets)
    int split;               // one-SM tiles: CTAs of a cluster that share a tile's k-blocks (1: no sharing)
    int wgrad;
    void* C;
    long long ldc, c_expert;
    int out_bf16;
    int vec;                 // rows of C are whole 16-byte pieces
    unsigned long long timeout_ns;
    unsigned int* status;
};

template <int BQ_, bool PAIR_, bool SWAP_, bool QVEC_>
struct Fp8Cfg {
    static constexpr int BQ = BQ_;
    static constexpr bool PAIR = PAIR_, SWAP = SWAP_, QVEC = QVEC_;   // QVEC: a scale for each row of Q
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int BP = 128 * CTAS;            // rows of P per tile
    static constexpr int BQL = BQ / CTAS;            // rows of Q that one CTA loads
    static constexpr int A_BYTES = 128 * 128;
    static constexpr int B_BYTES = BQL * 128;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = 4;
    static constexpr int PER_SM = SWAP ? 2 : 1;      // CTAs that fit on an SM
    static constexpr int NB = 512 / BQ < 8 ? 512 / BQ : 8;   // accumulators in tensor memory
    static constexpr int TMEM_COLS = NB * BQ;
    static constexpr int PW = SWAP ? 4 : 8;   // promotion warps, each 32 lanes × CW columns
    static constexpr int CW = BQ / (PW / 4);
    static constexpr int CHUNK = CW < 32 ? 16 : 32;   // columns per tensor-memory load
    static constexpr int THREADS = 128 + 32 * PW;
    // A finished tile of the unswapped form leaves through slabs of 32 rows × 128 bytes (16-byte
    // units permuted by the row, as the tensor copies do), SLABS of them per promotion warp
    static constexpr int SLABS = 2;
    static constexpr int SLAB_BYTES = 32 * 128;
    static constexpr int STORE_BYTES = SWAP ? 0 : PW * SLABS * SLAB_BYTES;
    // 128 sums per thread need more than the 168 registers a thread of 384 starts with: the
    // roles' warpgroup gives some of its own up (128·56 + 256·224 = 384·168)
    static constexpr bool SPLIT_REGS = CW > 64;
    static constexpr int SS = 8;                     // scale slots, a k-block each
    static constexpr int SLOT_Q = 128;               // a slot: P's scales, then Q's (each, or one per 128 rows)
    // Scales per column, many rows (QUAD): a thread holds two columns of every eight in four rows,
    // not all columns of one row, so that it reads a quarter of the columns' scales; those of the
    // four threads of a row lie QUAD_STEP apart, in four different groups of banks. (A broadcast
    // of 16 bytes takes shared memory as long as 128 bytes: with all columns to a thread the
    // scales' reads and the MMAs' own came to more than it gives.)
    static constexpr bool QUAD = QVEC && !SWAP;
    static constexpr int QUAD_STEP = CW / 4 + 4;
    static constexpr int SLOT = SLOT_Q + (QUAD ? 8 * QUAD_STEP : QVEC ? BQ : 4);
    static constexpr int TAB = kMaxExperts + 8;
    static constexpr int SUM_PITCH = BQ + 4;         // floats between rows of a shared tile's sums
    static constexpr int UR = 2;                     // units published ahead to the promotion warps
    static constexpr int NBARS = 2 * STAGES + 2 * SS + 2 * NB + 2 * UR + 1;
    static constexpr int SMEM_BYTES =
        1024 + STAGES * STAGE_BYTES + STORE_BYTES + SS * SLOT * 4 + 2 * TAB * 4 + UR * 32 + (NBARS + 4) * 8;
    static constexpr uint32_t IDESC = ptx::make_idesc(0, 0, 0, 0, BP, BQ);   // e4m3 both, K-major both
    static_assert(STAGE_BYTES % 1024 == 0 && SS * SLOT % 4 == 0, "16-byte aligned tables behind the slots");
    static_assert(PER_SM * (SMEM_BYTES + 1024) <= 233472 && PER_SM * TMEM_COLS <= 512, "CTAs of an SM");
    static_assert(128 * SUM_PITCH * 4 <= STAGES * STAGE_BYTES || PAIR, "a shared tile's sums fit the ring");
    static_assert(SMEM_BYTES <= 232448, "exceeds the 227 KB per-block shared memory limit");
    static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS >= 32 && TMEM_COLS <= 512, "TMEM columns");
    static_assert(BQ % 16 == 0 && CW % CHUNK == 0 && (CHUNK == 16 || CHUNK == 32), "column split");
};

// One output tile: its first row on either side, the rows that exist, the expert, and
// the k-blocks [kb0, kb0 + nk).
struct Fp8Unit {
    int p0, q0, p_end, q_end, e, kb0, nk;
};

// The tiles of all experts in one walk. first[e] counts the tiles before expert e;
// first[experts + 1] is the total (entry `experts` holds the rows behind the last one).
// For weight gradients first[] lists the experts by falling length instead.
template <class C>
__device__ __forceinline__ Fp8Unit fp8_unit(const Fp8Params& p, const int* first, const int* off, int u, int& cur) {
    Fp8Unit U;
    if (p.wgrad) {
        const int tp = (p.wrows + C::BP - 1) / C::BP, tq = (p.qrows + C::BQ - 1) / C::BQ;
        const int i = u / (tp * tq), r = u - i * (tp * tq);
        const int e = first[i];   // the experts by falling length
        U.e = e;
        U.p0 = r / tq * C::BP;
        U.q0 = r % tq * C::BQ;
        U.p_end = p.wrows;
        U.q_end = p.qrows;
        U.kb0 = off[e] >> 7;
        U.nk = (off[e + 1] >> 7) - U.kb0;
        return U;
    }
    while (u >= first[cur + 1]) ++cur;   // (u only grows along a CTA's walk)
    constexpr int TT = C::SWAP ? C::BQ : C::BP, TW = C::SWAP ? C::BP : C::BQ;
    constexpr int G = 8;                 // token tiles that share a pass over the weights
    const int tw = (p.wrows + TW - 1) / TW;
    const int t0 = off[cur], t_end = cur < p.experts ? off[cur + 1] : p.rows;
    const int tt = (t_end - t0 + TT - 1) / TT;
    const int v = u - first[cur];
    const int g = v / (G * tw) * G, gn = min(G, tt - g), r = v - g * tw;
    const int t = t0 + (g + r % gn) * TT, w = r / gn * TW;
    U.e = cur;
    U.kb0 = 0;
    U.nk = cur < p.experts ? p.num_kb : 0;
    U.p0 = C::SWAP ? w : t;
    U.q0 = C::SWAP ? t : w;
    U.p_end = C::SWAP ? p.wrows : t_end;
    U.q_end = C::SWAP ? t_end : p.wrows;
    return U;
}

template <int N>
__device__ __forceinline__ void fp8_tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
    if constexpr (N == 32)
        ptx::tmem_ld_32x32b_x32(addr, r);
    else
        ptx::tmem_ld_32x32b_x16(addr, r);
}

// Promotion of 32 (or 16) columns: sum += r · f, or r · (f · q[column]).
template <int N>
__device__ __forceinline__ void fp8_promote(uint64_t* sum, const uint32_t (&r)[N], float f) {
    const uint64_t ff = ptx::f32x2(f, f);
#pragma unroll
    for (int i = 0; i < N; i += 2) sum[i / 2] = ptx::fma_f32x2(ptx::f32x2(r[i], r[i + 1]), ff, sum[i / 2]);
}
template <int N>
__device__ __forceinline__ void fp8_promote(uint64_t* sum, const uint32_t (&r)[N], float f, const float* q) {
    const uint64_t ff = ptx::f32x2(f, f);
    const ulonglong2* q4 = reinterpret_cast<const ulonglong2*>(q);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const ulonglong2 qq = q4[i / 4];
        sum[i / 2] = ptx::fma_f32x2(ptx::f32x2(r[i], r[i + 1]), ptx::mul_f32x2(ff, qq.x), sum[i / 2]);
        sum[i / 2 + 1] = ptx::fma_f32x2(ptx::f32x2(r[i + 2], r[i + 3]), ptx::mul_f32x2(ff, qq.y), sum[i / 2 + 1]);
    }
}

// Stores a warp's 32 rows × CW columns (lane: row), a slab of 128 bytes of each row at a time.
// Whole slabs are copied out by the tensor copy engine while the warp goes on with the next
// tile (a tile's stores take longer than a k-block of its successor: waiting for them cost
// 12 % of a product with K = 4096 and a sixth of one with K = 2048); the map cuts columns
// behind the matrix off. A slab that an expert's end cuts, or whose rows do not start and end on
// whole 16-byte pieces, is read back and stored by the warp.
template <class C, typename T>
__device__ __forceinline__ void fp8_store_rows(const uint64_t (&sum)[C::CW / 2], uint8_t* slabs, int& used,
                                               const CUtensorMap* map, T* c, long long ldc, int row, int col, int e,
                                               int rows, int cols, bool vec, int lane) {
    constexpr int PER = 128 / sizeof(T), UNIT = 16 / sizeof(T);   // columns of a slab, of a 16-byte unit
    auto place = [](int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); };
    // (a copy rounds a row's end up to 16 bytes)
    const bool bulk = vec && rows >= 32, whole = cols % UNIT == 0;
#pragma unroll
    for (int c0 = 0; c0 < C::CW; c0 += PER) {
        uint8_t* slab = slabs + used * C::SLAB_BYTES;
        used = used + 1 == C::SLABS ? 0 : used + 1;
        if (lane == 0) ptx::bulk_wait_read<C::SLABS - 1>();   // the copy that last used this slab has read it
        __syncwarp();
        if constexpr (C::QUAD) {
#pragma unroll
            for (int g = 0; g < PER / 8; ++g)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 8 * k + lane / 4, col = g * 8 + lane % 4 * 2;
                    const float2 v = ptx::f32x2_get(sum[(c0 / 8 + g) * 4 + k]);
                    uint8_t* to = slab + place(r, col / UNIT) + col % UNIT * sizeof(T);
                    if constexpr (sizeof(T) == 2)
                        *reinterpret_cast<uint32_t*>(to) = pack_bf16(v.x, v.y);
                    else
                        *reinterpret_cast<float2*>(to) = v;
                }
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                uint4 v;
                const uint64_t* s = sum + (c0 + u * UNIT) / 2;
                if constexpr (sizeof(T) == 2) {
                    const float2 a = ptx::f32x2_get(s[0]), b = ptx::f32x2_get(s[1]), d = ptx::f32x2_get(s[2]),
                                 e4 = ptx::f32x2_get(s[3]);
                    v = make_uint4(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y), pack_bf16(d.x, d.y), pack_bf16(e4.x, e4.y));
                } else {
                    const float2 a = ptx::f32x2_get(s[0]), b = ptx::f32x2_get(s[1]);
                    v = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
                }
                *reinterpret_cast<uint4*>(slab + place(lane, u)) = v;
            }
        }
        if (bulk && (whole || c0 + PER <= cols)) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (c0 < cols) ptx::tma_store_3d(map, ptx::smem_u32(slab), col + c0, row, e);
                ptx::bulk_commit();
            }
            continue;
        }
        __syncwarp();
        if (vec) {   // 16-byte pieces, four rows to an instruction
            const int u = lane & 7, n = cols - c0 - u * UNIT;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = k * 4 + (lane >> 3);
                const T* from = reinterpret_cast<const T*>(slab + place(r, u));
                T* to = c + r * ldc + c0 + u * UNIT;
                if (r >= rows) continue;
                if (n >= UNIT) {
                    *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
                } else {
#pragma unroll
                    for (int i = 0; i < UNIT; ++i)
                        if (i < n) to[i] = from[i];
                }
            }
        } else {   // rows at any address: an element a lane, a row at a time
#pragma unroll 4
            for (int r = 0; r < min(rows, 32); ++r) {
#pragma unroll
                for (int i = lane; i < PER; i += 32)
                    if (c0 + i < cols)
                        c[r * ldc + c0 + i] = reinterpret_cast<const T*>(slab + place(r, i / UNIT))[i % UNIT];
            }
        }
        __syncwarp();
        if (lane == 0) ptx::bulk_commit();   // (an empty group: every slab used counts as one)
    }
}

template <int BQ, bool PAIR, bool SWAP, bool QVEC>
__global__ void __launch_bounds__(Fp8Cfg<BQ, PAIR, SWAP, QVEC>::THREADS, Fp8Cfg<BQ, PAIR, SWAP, QVEC>::PER_SM)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmC, const Fp8Params p) {
    using C = Fp8Cfg<BQ, PAIR, SWAP, QVEC>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = ptx::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    uint8_t* slabs = smem + C::STAGES * C::STAGE_BYTES;
    float* slots = reinterpret_cast<float*>(slabs + C::STORE_BYTES);
    int* published = reinterpret_cast<int*>(slots + C::SS * C::SLOT);   // UR × 8, 16-byte aligned
    uint64_t* bars = reinterpret_cast<uint64_t*>(published + C::UR * 8);
    int* first = reinterpret_cast<int*>(bars + C::NBARS + 2);
    int* off = first + C::TAB;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::NBARS);
    volatile uint32_t* abort_flag = tmem_holder + 1;
    volatile uint32_t* bad_offsets = tmem_holder + 2;

    const uint32_t full0 = ptx::smem_u32(bars);
    const uint32_t empty0 = full0 + 8 * C::STAGES;
    const uint32_t sfull0 = empty0 + 8 * C::STAGES;
    const uint32_t sempty0 = sfull0 + 8 * C::SS;
    const uint32_t accf0 = sempty0 + 8 * C::SS;
    const uint32_t acce0 = accf0 + 8 * C::NB;
    const uint32_t ufull0 = acce0 + 8 * C::NB;
    const uint32_t uempty0 = ufull0 + 8 * C::UR;
    const uint32_t drain_bar = uempty0 + 8 * C::UR;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(full0 + 8 * s, 1);     // the (leader's) producer and the bytes
            ptx::mbar_init(empty0 + 8 * s, 1);    // the MMAs' commit
        }
        for (int s = 0; s < C::SS; ++s) {
            ptx::mbar_init(sfull0 + 8 * s, 64);   // the scale warps' lanes
            ptx::mbar_init(sempty0 + 8 * s, C::PW);
        }
        for (int b = 0; b < C::NB; ++b) {
            ptx::mbar_init(accf0 + 8 * b, 1);
            ptx::mbar_init(acce0 + 8 * b, C::CTAS * C::PW);
        }
        for (int i = 0; i < C::UR; ++i) {
            ptx::mbar_init(ufull0 + 8 * i, 1);
            ptx::mbar_init(uempty0 + 8 * i, C::PW);
        }
        ptx::mbar_init(drain_bar, 1);
        *abort_flag = 0u;
        *bad_offsets = 0u;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmP);
        ptx::prefetch_tensormap(&tmQ);
        if (!SWAP && p.vec) ptx::prefetch_tensormap(&tmC);
    }
    if (warp == 3) {
        if constexpr (PAIR) {
            ptx::tmem_alloc_pair(ptx::smem_u32(tmem_holder), C::TMEM_COLS);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_u32(tmem_holder), C::TMEM_COLS);
            ptx::tmem_relinquish();
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    if constexpr (PAIR)
        ptx::cluster_sync();
    else
        __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    // nothing above touches global memory; the offsets, operands and scales may be the
    // previous kernel's results
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // the experts' rows and the running count of their tiles
    const int E = p.experts;
    for (int e = threadIdx.x; e <= E; e += C::THREADS) {
        const int lo = p.offsets ? p.offsets[e] : (e == 0 ? 0 : p.rows);
        const int hi = e == E ? p.rows : p.offsets ? p.offsets[e + 1] : p.rows;
        off[e] = lo;
        if (lo < 0 || lo > hi || hi > p.rows || (e == 0 && lo != 0) || (p.wgrad && (lo & 127))) *bad_offsets = 1u;
    }
    __syncthreads();
    int units = 0;
    if (*bad_offsets) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0u, static_cast<unsigned int>(DEV_BAD_OFFSETS));
    } else if (p.wgrad) {
        // a tile takes as long as its expert has rows: long ones first, dealt out back and forth
        units = E * ((p.wrows + C::BP - 1) / C::BP) * ((p.qrows + BQ - 1) / BQ);
        for (int e = threadIdx.x; e < E; e += C::THREADS) {
            const int mine = off[e + 1] - off[e];
            int before = 0;
            if (E <= kMaxSorted) {
                for (int o = 0; o < E; ++o) {
                    const int n = off[o + 1] - off[o];
                    before += n > mine || (n == mine && o < e);
                }
            }
            first[E <= kMaxSorted ? before : e] = e;
        }
        __syncthreads();   // (uniform: every thread takes this branch)
    } else {
        constexpr int TT = SWAP ? BQ : C::BP, TW = SWAP ? C::BP : BQ;
        const int tw = (p.wrows + TW - 1) / TW;
        if (warp == 0) {
            int run = 0;
            for (int e0 = 0; e0 <= E; e0 += 32) {
                const int e = e0 + lane;
                int n = 0;
                if (e <= E) n = ((e < E ? off[e + 1] : p.rows) - off[e] + TT - 1) / TT * tw;
                int inc = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, inc, d);
                    if (lane >= d) inc += o;
                }
                if (e <= E) first[e + 1] = run + inc;
                run += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0) first[0] = 0;
        }
        __syncthreads();   // (uniform: every thread takes this branch)
        units = first[E + 1];
    }
    const int share = PAIR ? C::CTAS : p.split;   // CTAs that work on one tile
    const int u0 = blockIdx.x / share, ustep = gridDim.x / share;
    // this CTA's part of a tile's k-blocks
    [[maybe_unused]] const int part = PAIR ? 0 : static_cast<int>(blockIdx.x) % share;
    // step j of this CTA's walk
    auto walk = [&](int j) {
        if (QVEC && !SWAP && p.wgrad && (j & 1)) return (j + 1) * ustep - 1 - u0;
        return j * ustep + u0;
    };
    auto unit = [&](int u, int& cur) {
        Fp8Unit U = fp8_unit<C>(p, first, off, u, cur);
        if constexpr (!PAIR) {
            const int n = U.nk, lo = part * n / share;
            U.kb0 += lo;
            U.nk = (part + 1) * n / share - lo;
        }
        return U;
    };
    [[maybe_unused]] const AbortNet net{ptx::smem_u32(const_cast<uint32_t*>(abort_flag)), C::CTAS};
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned int code) {
        if constexpr (PAIR)
            return wait_warp_pair(bar, parity, abort_flag, net, p.timeout_ns, p.status, code);
        else
            return wait_warp(bar, parity, abort_flag, p.timeout_ns, p.status, code);
    };

    if (warp < 4) {
        if constexpr (C::SPLIT_REGS) ptx::setmaxnreg_dec<56>();
        if (warp == 0) {
            // ------------------------------------------------ operand loads
            const uint32_t full_leader0 = PAIR ? ptx::mapa_shared(full0, 0u) : full0;
            uint32_t s = 0, ph = 0;
            int cur = 0;
            bool ok = true;
            for (int j = 0, u = u0; ok && u < units; u = walk(++j)) {
                const Fp8Unit U = unit(u, cur);
                const int pe = (SWAP && !p.wgrad) ? U.e : 0, qe = (!SWAP && !p.wgrad) ? U.e : 0;
                const int prow = U.p0 + static_cast<int>(rank) * 128, qrow = U.q0 + static_cast<int>(rank) * C::BQL;
                for (int kb = 0; kb < U.nk; ++kb) {
                    if (!wait(empty0 + 8 * s, ph ^ 1u, DEV_TIMEOUT_PRODUCER)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = ptx::smem_u32(smem) + s * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                    const int x = (U.kb0 + kb) * 128;
                    if (rank == 0) ptx::mbar_arrive_expect_tx_elected(full0 + 8 * s, C::CTAS * C::STAGE_BYTES);
                    if constexpr (PAIR) {
                        ptx::tma_load_3d_pair_elected(sa, &tmP, full_leader0 + 8 * s, x, prow, pe);
                        ptx::tma_load_3d_pair_elected(sb, &tmQ, full_leader0 + 8 * s, x, qrow, qe);
                    } else {
                        ptx::tma_load_3d_elected(sa, &tmP, full0 + 8 * s, x, prow, pe);
                        ptx::tma_load_3d_elected(sb, &tmQ, full0 + 8 * s, x, qrow, qe);
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
            // ------------------------------------------------ MMA issue (a pair's leader)
            if (rank == 0) {
                const uint32_t stage0 = ptx::smem_u32(smem);
                const uint64_t adesc0 = ptx::sdesc_sw128(stage0, 16, 1024);
                const uint64_t bdesc0 = ptx::sdesc_sw128(stage0 + C::A_BYTES, 16, 1024);
                constexpr uint64_t STEP = C::STAGE_BYTES / 16;
                uint32_t s = 0, ph = 0, b = 0, bph = 0;
                int cur = 0;
                bool ok = true;
                for (int j = 0, u = u0; ok && u < units; u = walk(++j)) {
                    const Fp8Unit U = unit(u, cur);
                    for (int kb = 0; kb < U.nk; ++kb) {
                        // (the operands are there long before the accumulator is free)
                        if (!wait(full0 + 8 * s, ph, DEV_TIMEOUT_MMA_FULL) ||
                            !wait(acce0 + 8 * b, bph ^ 1u, DEV_TIMEOUT_MMA_ACC)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        const uint64_t ad = adesc0 + s * STEP, bd = bdesc0 + s * STEP;
                        const uint32_t d = tmem_base + b * BQ;
                        if constexpr (PAIR) {
                            ptx::mma_f8_pair_x4_elected(d, ad, bd, ad + 2, bd + 2, ad + 4, bd + 4, ad + 6, bd + 6,
                                                        C::IDESC, 0u);
                            ptx::mma_commit_pair_multicast_elected(empty0 + 8 * s, 0x3);
                            ptx::mma_commit_pair_multicast_elected(accf0 + 8 * b, 0x3);
                        } else {
                            ptx::mma_f8_x4_elected(d, ad, bd, ad + 2, bd + 2, ad + 4, bd + 4, ad + 6, bd + 6, C::IDESC,
                                                   0u);
                            ptx::mma_commit_elected(empty0 + 8 * s);
                            ptx::mma_commit_elected(accf0 + 8 * b);
                        }
                        if (++s == C::STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
                        if (++b == C::NB) {
                            b = 0;
                            bph ^= 1u;
                        }
                    }
                }
                if (!ok) {
                    if constexpr (PAIR)
                        ptx::mma_commit_pair_multicast_elected(drain_bar, 0x1);
                    else
                        ptx::mma_commit_elected(drain_bar);
                    if (lane == 0) wait_drain(drain_bar, 0, p.timeout_ns);
                }
            }
            __syncwarp();
        } else {
            // ------------------------------------------------ scales: warp 2 P's, warp 3 Q's
            constexpr int NI = QVEC && BQ > 128 ? BQ / 32 : 4;
            const bool of_p = warp == 2;
            const Fp8Side& side = of_p ? p.P : p.Q;
            const int per = of_p ? (p.P.block ? 1 : 128) : QVEC ? BQ : (BQ + 127) / 128;   // scales of a k-block
            const long long step = 32 * side.s_row;
            const bool quad = C::QUAD && !of_p;
            const int place0 = of_p ? lane
                               : quad ? C::SLOT_Q + (lane & 7) / 2 * C::QUAD_STEP + (lane >> 3) * 2 + (lane & 1)
                                      : C::SLOT_Q + lane;
            const uint32_t dst0 = ptx::smem_u32(slots) + 4 * place0;
            uint32_t s = 0, ph = 0;
            int cur = 0;
            bool ok = true;
            for (int j = 0, u = u0; ok && u < units; u = walk(++j)) {
                const Fp8Unit U = unit(u, cur);
                if (of_p) {   // what the promotion warps need of it (working it out would hold them up between tiles)
                    if (!wait(uempty0 + 8 * (j % C::UR), (j / C::UR & 1) ^ 1u, DEV_TIMEOUT_PRODUCER)) break;
                    if (lane == 0) {
                        int4* to = reinterpret_cast<int4*>(published + 8 * (j % C::UR));
                        to[0] = make_int4(U.p0, U.q0, U.p_end, U.q_end);
                        to[1] = make_int4(U.e, U.nk, 0, 0);
                        ptx::mbar_arrive(ufull0 + 8 * (j % C::UR));
                    }
                    __syncwarp();
                }
                const int row0 = of_p ? U.p0 + static_cast<int>(rank) * 128 : U.q0, end = of_p ? U.p_end : U.q_end;
                const int r0 = side.block ? row0 >> 7 : row0;
                const int n = min(per, (side.block ? (end + 127) >> 7 : end) - r0);   // those that exist; zeros behind them
                const float* at = side.scale + (of_p == SWAP ? U.e * side.s_expert : 0ll) + U.kb0 * side.s_group +
                                  (r0 + lane) * side.s_row;
                for (int kb = 0; kb < U.nk; ++kb, at += side.s_group) {
                    if (!wait(sempty0 + 8 * s, ph ^ 1u, DEV_TIMEOUT_PRODUCER)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const bool in = lane + 32 * i < n;
                        // (QUAD: 32 columns are four groups of eight, a thread's share of CW columns one run)
                        const int step_i = quad ? 32 * i / C::CW * 4 * C::QUAD_STEP + 32 * i % C::CW / 4 : 32 * i;
                        if (lane + 32 * i < per)
                            ptx::cp_async_4(dst0 + 4 * (s * C::SLOT + step_i), in ? at + i * step : side.scale, in ? 4u : 0u);
                    }
                    ptx::cp_async_arrive_noinc(sfull0 + 8 * s);
                    if (++s == C::SS) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            ptx::cp_async_wait_all();
            __syncwarp();
        }
    } else {
        if constexpr (C::SPLIT_REGS) ptx::setmaxnreg_inc<224>();
        // ------------------------------------------------ promotion and stores
        const int quarter = warp & 3;            // the tensor-memory lanes this warp may read
        const int h = (warp - 4) >> 2;           // its share of the columns
        const int prl = quarter * 32 + lane;
        const uint32_t acce_leader0 = PAIR ? ptx::mapa_shared(acce0, 0u) : acce0;
        uint32_t s = 0, ph = 0, b = 0, bph = 0;
        [[maybe_unused]] int used = 0;   // the slab whose turn it is
        bool ok = true;
        for (int j = 0, u = u0; ok && u < units; u = walk(++j)) {
            uint64_t sum[C::CW / 2];   // two columns each
#pragma unroll
            for (int i = 0; i < C::CW / 2; ++i) sum[i] = 0;
            const int* mine = published + 8 * (j % C::UR);
            if (!wait(ufull0 + 8 * (j % C::UR), j / C::UR & 1, DEV_TIMEOUT_EPILOGUE)) break;
            const int nk = mine[5];
            for (int kb = 0; kb < nk; ++kb) {
                if (!wait(sfull0 + 8 * s, ph, DEV_TIMEOUT_EPILOGUE)) {
                    ok = false;
                    break;
                }
                const float* slot = slots + s * C::SLOT;
                [[maybe_unused]] float f = slot[p.P.block ? 0 : prl];
                if constexpr (!QVEC) f *= slot[C::SLOT_Q + ((h * C::CW) >> 7)];
                if (!wait(accf0 + 8 * b, bph, DEV_TIMEOUT_EPILOGUE)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                auto release = [&]() {   // the accumulator is read: free for the next k-block
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (PAIR)
                            ptx::mbar_arrive_cluster_relaxed(acce_leader0 + 8 * b);
                        else
                            ptx::mbar_arrive_relaxed(acce0 + 8 * b);
                    }
                };
                const uint32_t t = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + b * BQ + h * C::CW;
                if constexpr (C::QUAD) {
                    float rows[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) rows[k] = slot[quarter * 32 + 8 * k + lane / 4];
                    const ulonglong2* q2 =
                        reinterpret_cast<const ulonglong2*>(slot + C::SLOT_Q + (4 * h + lane % 4) * C::QUAD_STEP);
#pragma unroll
                    for (int c = 0; c < C::CW; c += 32) {
                        const ulonglong2 qa = q2[c / 16], qb = q2[c / 16 + 1];
                        const uint64_t q[4] = {qa.x, qa.y, qb.x, qb.y};
#pragma unroll
                        for (int k = 0; k < 4; k += 2) {   // the lower and the upper sixteen lanes
                            uint32_t r[16];
                            ptx::tmem_ld_16x256b_x4(t + (static_cast<uint32_t>(k * 8) << 16) + c, r);
                            ptx::tmem_ld_wait(r);
                            if (c + 32 == C::CW && k == 2) release();
                            const uint64_t fa = ptx::f32x2(rows[k], rows[k]), fb = ptx::f32x2(rows[k + 1], rows[k + 1]);
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                uint64_t* to = sum + (c / 8 + g) * 4 + k;
                                to[0] = ptx::fma_f32x2(ptx::f32x2(r[4 * g], r[4 * g + 1]), ptx::mul_f32x2(fa, q[g]), to[0]);
                                to[1] = ptx::fma_f32x2(ptx::f32x2(r[4 * g + 2], r[4 * g + 3]), ptx::mul_f32x2(fb, q[g]),
                                                       to[1]);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < C::CW; c += C::CHUNK) {
                        uint32_t r[C::CHUNK];
                        fp8_tmem_ld<C::CHUNK>(t + c, r);
                        ptx::tmem_ld_wait(r);
                        if (c + C::CHUNK == C::CW) release();
                        if constexpr (QVEC)
                            fp8_promote<C::CHUNK>(sum + c / 2, r, f, slot + C::SLOT_Q + c);
                        else
                            fp8_promote<C::CHUNK>(sum + c / 2, r, f);
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sempty0 + 8 * s);
                if (++s == C::SS) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++b == C::NB) {
                    b = 0;
                    bph ^= 1u;
                }
            }
            if (!ok) break;
            // (read only now: the sums leave few registers)
            const int4 u4 = *reinterpret_cast<const int4*>(mine);
            const Fp8Unit U = {u4.x, u4.y, u4.z, u4.w, mine[4], 0, nk};
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(uempty0 + 8 * (j % C::UR));
            const int qc = U.q0 + h * C::CW;
            if constexpr (SWAP) {
                // consecutive lanes hold consecutive columns of C
                const int pr = U.p0 + prl;
                const int n = pr < U.p_end ? min(C::CW, U.q_end - qc) : 0;
                const long long at = static_cast<long long>(qc) * p.ldc + pr;
                // (the ring is free: a shared tile is this CTA's only one, and all its MMAs are done)
                float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
                for (int i = 0; i < C::CW; ++i) {
                    const float2 v2 = ptx::f32x2_get(sum[i / 2]);
                    const float v = i & 1 ? v2.y : v2.x;
                    if (share > 1) {
                        sums[(h * C::CW + i) * 128 + prl] = v;
                    } else if (i < n) {
                        if (p.out_bf16)
                            static_cast<__nv_bfloat16*>(p.C)[at + i * p.ldc] = __float2bfloat16_rn(v);
                        else
                            static_cast<float*>(p.C)[at + i * p.ldc] = v;
                    }
                }
            } else {
                const int pw = U.p0 + static_cast<int>(rank) * 128 + quarter * 32;   // this warp's first row
                const int rows = U.p_end - pw, cols = U.q_end - qc;
                const long long at = (p.wgrad ? U.e * p.c_expert : 0ll) + static_cast<long long>(pw) * p.ldc + qc;
                uint8_t* slab = slabs + (warp - 4) * C::SLABS * C::SLAB_BYTES;
                if (C::QUAD && !PAIR && share > 1) {
                    float* to = reinterpret_cast<float*>(smem) + h * C::CW + lane % 4 * 2;
#pragma unroll
                    for (int i = 0; i < C::CW / 2; ++i)
                        *reinterpret_cast<float2*>(to + (quarter * 32 + i % 4 * 8 + lane / 4) * C::SUM_PITCH + i / 4 * 8) =
                            ptx::f32x2_get(sum[i]);
                } else if (!PAIR && share > 1) {
                    float4* to = reinterpret_cast<float4*>(reinterpret_cast<float*>(smem) + prl * C::SUM_PITCH + h * C::CW);
#pragma unroll
                    for (int i = 0; i < C::CW; i += 4) {
                        const float2 x = ptx::f32x2_get(sum[i / 2]), y = ptx::f32x2_get(sum[i / 2 + 1]);
                        to[i / 4] = make_float4(x.x, x.y, y.x, y.y);
                    }
                } else if (rows > 0 && cols > 0) {
                    const int e = p.wgrad ? U.e : 0;
                    if (p.out_bf16)
                        fp8_store_rows<C>(sum, slab, used, &tmC, static_cast<__nv_bfloat16*>(p.C) + at, p.ldc, pw, qc, e,
                                          rows, cols, p.vec != 0, lane);
                    else
                        fp8_store_rows<C>(sum, slab, used, &tmC, static_cast<float*>(p.C) + at, p.ldc, pw, qc, e, rows,
                                          cols, p.vec != 0, lane);
                }
            }
            __syncwarp();
        }
        if (!SWAP && lane == 0) ptx::bulk_wait<0>();
        __syncwarp();
    }

    // ------------------------------------------------ shared tiles: the parts' sums, in their order
    if (!PAIR && share > 1) {
        __syncwarp();
        ptx::cluster_sync();   // every part's sums are in its shared memory
        if (warp >= 4 && u0 < units) {
            int cur = 0;
            const Fp8Unit U = fp8_unit<C>(p, first, off, u0, cur);
            const uint32_t sums = ptx::smem_u32(smem);
            if constexpr (SWAP) {
                const int prl = (warp & 3) * 32 + lane, pr = U.p0 + prl;
                for (int i = part; i < BQ; i += share) {
                    if (pr >= U.p_end || U.q0 + i >= U.q_end) continue;
                    float v = 0.0f;
                    for (int r = 0; r < share; ++r)
                        v += ptx::ld_cluster_f32(ptx::mapa_shared(sums + 4 * (i * 128 + prl), static_cast<uint32_t>(r)));
                    const long long at = static_cast<long long>(U.q0 + i) * p.ldc + pr;
                    if (p.out_bf16)
                        static_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(v);
                    else
                        static_cast<float*>(p.C)[at] = v;
                }
            } else {
                // a warp a row, a lane four columns
                const int n = U.q_end - U.q0 - lane * 4;
                for (int i = part + share * (warp - 4); i < 128; i += share * C::PW) {
                    if (U.p0 + i >= U.p_end || n <= 0) continue;
                    float v[4] = {};
                    for (int r = 0; r < share; ++r) {
                        const uint4 x = ptx::ld_cluster_v4(
                            ptx::mapa_shared(sums + 4 * (i * C::SUM_PITCH + lane * 4), static_cast<uint32_t>(r)));
                        v[0] += __uint_as_float(x.x);
                        v[1] += __uint_as_float(x.y);
                        v[2] += __uint_as_float(x.z);
                        v[3] += __uint_as_float(x.w);
                    }
                    const long long at = (p.wgrad ? U.e * p.c_expert : 0ll) +
                                         static_cast<long long>(U.p0 + i) * p.ldc + U.q0 + lane * 4;
                    if (p.out_bf16) {
                        __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.C) + at;
                        if (p.vec && n >= 4) {
                            *reinterpret_cast<uint2*>(c) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k < n) c[k] = __float2bfloat16_rn(v[k]);
                        }
                    } else {
                        float* c = static_cast<float*>(p.C) + at;
                        if (p.vec && n >= 4) {
                            *reinterpret_cast<float4*>(c) = make_float4(v[0], v[1], v[2], v[3]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k < n) c[k] = v[k];
                        }
                    }
                }
            }
        }
        __syncwarp();
        ptx::cluster_sync();   // no part leaves while another may still read its sums
    }

    // ------------------------------------------------ teardown
    ptx::tc_fence_before();
    if constexpr (PAIR)
        ptx::cluster_sync();   // no CTA frees TMEM or exits while its peer may still signal it
    else
        __syncthreads();
    if (warp == 3) {
        ptx::tc_fence_after();
        if constexpr (PAIR)
            ptx::tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
        else
            ptx::tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace tcl
