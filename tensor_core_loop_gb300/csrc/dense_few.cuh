// Products of few rows of tokens with bf16 weight matrices: D = x·W^T, x T × K with T <= 128.
//
// What bounds them is the weights' way from HBM, once: 128 weight rows are the MMA's M side
// (tensor-memory lanes), the tokens its N side, so that no shared memory and no MMA is spent on
// tokens that do not exist and a thread holds one output column of every token. The loads run
// through a ring of 64-value k-blocks, whose slots have room for 128 weight rows: 184 to 209 KB are in flight on
// each SM where a tile has as many, 102 to 147 KB with 64 rows. A tile has as many
// weight rows (128 at most) as give all SMs the same share; where there are too few rows
// for that, the CTAs of a cluster share a tile's k-blocks and one after another's sums are
// added over distributed shared memory.
//
// The ends are those of dense_product.cuh (what they round to bf16, and why, stands there), for the forward direction: STORE, GATE (two weight
// tiles to a CTA: 128 rows of either matrix), ENTROPY (sums over all vocabulary rows that a warp saw).
#pragma once

#include "dense_product.cuh"

namespace tcl {

struct DenseFewParams {
    int T, N, num_kb, tiles, split;
    int rows;              // weight rows of a tile, a multiple of 8: as many as deal them out evenly (128 at most)
    int act;
    int early;             // the weights are not what the kernel before this one in the stream writes
    DenseOut out[3];
    const void* targets;
    int wide_targets;
    float2* parts;         // ENTROPY: [warp, four to a CTA][token]
    float* target_logit;
    unsigned long long timeout_ns;
    unsigned int* status;
};

// f(0), f(1), ... f(N - 1) with the numbers as types.
template <int N, class F>
__device__ __forceinline__ void dense_each(F f) {
    if constexpr (N > 0) {
        dense_each<N - 1>(f);
        f(std::integral_constant<int, N - 1>());
    }
}

template <int BQ_, DenseEnd E_>
struct DenseFewCfg {
    static constexpr int BQ = BQ_;                       // tokens
    static constexpr int MATS = E_ == DenseEnd::GATE ? 2 : 1;
    static constexpr int A_BYTES = 128 * 128, Q_BYTES = BQ * 128;
    static constexpr int STAGE_BYTES = MATS * A_BYTES + Q_BYTES;
    static constexpr int STAGES = 212992 / STAGE_BYTES;
    // ENTROPY: a tile's k-blocks go to several accumulators in turn, which are added in the end. The tensor core
    // truncates its fp32 sums, so the fewer additions to one the better: with K = 4096 and four of them the
    // log-sum-exp of 16 tokens is off by 1.7e-7 of its norm instead of 7.5e-7, in the same time.
    static constexpr int CHAINS = E_ != DenseEnd::ENTROPY ? 1 : BQ <= 64 ? 4 : 2;
    static constexpr int COLS = MATS * CHAINS * BQ;      // tensor-memory columns of a tile
    static constexpr int TMEM_COLS = 2 * COLS < 32 ? 32 : 2 * COLS;
    static constexpr int THREADS = 64 + 128;
    static constexpr int NBARS = 2 * STAGES + 5;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + (NBARS + 2) * 8;
    static_assert(SMEM_BYTES <= 232448 && TMEM_COLS <= 512, "fits an SM");
    static_assert(MATS * BQ * 128 * 4 <= STAGES * STAGE_BYTES, "a shared tile's sums fit the ring");
    static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0, "tensor-memory columns");
};

// k-blocks of 64 values: four MMAs each, one or two weight tiles.
template <int BQ, DenseEnd E>
__global__ void __launch_bounds__(DenseFewCfg<BQ, E>::THREADS, 1)
    dense_few_kernel(const __grid_constant__ CUtensorMap tmW0, const __grid_constant__ CUtensorMap tmW1,
                     const __grid_constant__ CUtensorMap tmX, const DenseFewParams p) {
    using C = DenseFewCfg<BQ, E>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = ptx::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE_BYTES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::NBARS);
    volatile uint32_t* abort_flag = tmem_holder + 1;

    const uint32_t full0 = ptx::smem_u32(bars);
    const uint32_t empty0 = full0 + 8 * C::STAGES;
    const uint32_t accf0 = empty0 + 8 * C::STAGES;
    const uint32_t acce0 = accf0 + 16;
    const uint32_t drain_bar = acce0 + 16;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(full0 + 8 * s, 1);
            ptx::mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(accf0 + 8 * b, 1);
            ptx::mbar_init(acce0 + 8 * b, 4);
        }
        ptx::mbar_init(drain_bar, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmW0);
        ptx::prefetch_tensormap(&tmX);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_holder), C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    const int share = p.split;
    const int u0 = blockIdx.x / share, ustep = gridDim.x / share, part = static_cast<int>(blockIdx.x) % share;
    const int lo = static_cast<int>(static_cast<long long>(p.num_kb) * part / share);
    const int hi = static_cast<int>(static_cast<long long>(p.num_kb) * (part + 1) / share);
    // The weights of the first k-blocks, up to a ring of them, are on their way before the kernel before this
    // one has ended, where that kernel does not write them.
    const int ahead = p.early && u0 < p.tiles ? min(hi - lo, C::STAGES) : 0;
    auto load_weights = [&](uint32_t s, int kb, int tile) {
        const uint32_t sa = ptx::smem_u32(smem) + s * C::STAGE_BYTES, fb = full0 + 8 * s;
        ptx::mbar_arrive_expect_tx_elected(fb, C::MATS * p.rows * 128 + C::Q_BYTES);
        ptx::tma_load_2d_elected(sa, &tmW0, fb, kb * 64, tile * p.rows);
        if constexpr (C::MATS == 2) ptx::tma_load_2d_elected(sa + C::A_BYTES, &tmW1, fb, kb * 64, tile * p.rows);
    };
    if (warp == 0)
        for (int i = 0; i < ahead; ++i) load_weights(i, lo + i, u0);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned int code) {
        return wait_warp(bar, parity, abort_flag, p.timeout_ns, p.status, code);
    };
    // ENTROPY: what this warp has summed up over its tiles, and the rows of W that are the tokens' targets (-1:
    // none); lane 2j (and 2j + 1) holds those of the tokens j, 16 + j, 32 + j, ...
    constexpr int SLOTS = E == DenseEnd::ENTROPY ? BQ / 16 : 1;
    [[maybe_unused]] float run_ref[SLOTS] = {}, run_sum[SLOTS] = {};
    [[maybe_unused]] int target[SLOTS];
    if constexpr (E == DenseEnd::ENTROPY) {
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) {
            const int i = 16 * k + lane / 2;
            const long long t = i >= p.T           ? -1
                                : p.wide_targets ? static_cast<const long long*>(p.targets)[i]
                                                 : static_cast<const int*>(p.targets)[i];
            target[k] = t >= 0 && t < p.N ? static_cast<int>(t) : -1;
        }
    }
    // One token's logits, the first `there` of v in each lane: their exponentials' sum, relative to the largest of
    // them if need be.
    [[maybe_unused]] auto one_token = [&](const auto& v, int there, float& ref, float& sum) {
        constexpr int N = sizeof(v) / sizeof(v[0]);
        auto total = [&](float taken) {
            float x = 0.0f;
#pragma unroll
            for (int k = 0; k < N; ++k) x += k < there ? ptx::exp2_approx(fmaf(v[k], 1.4426950408889634f, -taken)) : 0.0f;
#pragma unroll
            for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            return x;
        };
        ref = 0.0f;
        sum = total(0.0f);
        if (dense_plain_sum(sum)) return;
        float top = __int_as_float(0xff800000);
#pragma unroll
        for (int k = 0; k < N; ++k) top = k < there ? fmaxf(top, v[k]) : top;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        ref = dense_exponent(top);
        sum = total(ref);
    };
    // Sixteen tokens' logits (16k ..) of this lane's row. Each step of the butterfly halves the tokens that a lane
    // adds up: 16 shuffles for 16 sums over 32 lanes.
    [[maybe_unused]] auto sixteen = [&](int tile, auto slot, const uint32_t (&r)[16]) {
        constexpr int k = decltype(slot)::value;
        const int in_tile = (warp & 3) * 32 + lane, row0 = tile * p.rows + (warp & 3) * 32, row = row0 + lane;
        if (row0 >= p.N || (warp & 3) * 32 >= p.rows || 16 * k >= p.T) return;   // (the same for all lanes)
        const bool in = in_tile < p.rows && row < p.N;
        if (__any_sync(0xffffffffu, target[k] >= row0 && target[k] < row0 + 32)) {
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
                const int t = __shfl_sync(0xffffffffu, target[k], 2 * i);
                if (in && row == t) {
                    float v = 0.0f;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j == i) v = __uint_as_float(r[j]);
                    p.target_logit[16 * k + i] = v;
                }
            }
        }
        float e[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] = in ? ptx::exp2_approx(__uint_as_float(r[i]) * 1.4426950408889634f) : 0.0f;
        auto halve = [&](auto half) {
            constexpr int n = decltype(half)::value;
            const bool upper = lane & (2 * n);
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float given = __shfl_xor_sync(0xffffffffu, upper ? e[i] : e[i + n], 2 * n);
                e[i] = (upper ? e[i + n] : e[i]) + given;
            }
        };
        halve(std::integral_constant<int, 8>());
        halve(std::integral_constant<int, 4>());
        halve(std::integral_constant<int, 2>());
        halve(std::integral_constant<int, 1>());
        e[0] += __shfl_xor_sync(0xffffffffu, e[0], 1);
        const bool exists = 16 * k + lane / 2 < p.T;
        if (!__any_sync(0xffffffffu, exists && !dense_plain_sum(e[0]))) {
            dense_merge(run_ref[k], run_sum[k], 0.0f, e[0]);
            return;
        }
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
            float v[1] = {0.0f}, ref, sum;
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j == i) v[0] = __uint_as_float(r[j]);
            one_token(v, in ? 1 : 0, ref, sum);
            if (lane / 2 == i) dense_merge(run_ref[k], run_sum[k], ref, sum);
        }
    };
    // STORE, GATE: 16 tokens' results (from token c on) of this lane's row; consecutive lanes hold consecutive columns
    [[maybe_unused]] auto column = [&](int tile, int c, const uint32_t (&r)[16], const uint32_t (&r1)[16]) {
        // (the lanes behind the tile's rows hold what the ring held before)
        const int in_tile = (warp & 3) * 32 + lane, row = tile * p.rows + in_tile, n = p.T - c;
        if (in_tile >= p.rows || row >= p.N) return;
        auto put = [&](const DenseOut& o, const auto& x) {
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(o.p) + c * o.ld + row;
#pragma unroll
            for (int i = 0; i < 16; ++i, to += o.ld)
                if (i < n) *to = __float2bfloat16_rn(x(i));
        };
        if constexpr (E == DenseEnd::GATE) {
            dense_with_act(p.act, [&](auto act) {
                put(p.out[0], [&](int i) {
                    float unused;
                    return dense_act<decltype(act)::value, false>(__uint_as_float(r[i]), unused) * __uint_as_float(r1[i]);
                });
            });
            if (p.out[1].p) {
                put(p.out[1], [&](int i) { return __uint_as_float(r[i]); });
                put(p.out[2], [&](int i) { return __uint_as_float(r1[i]); });
            }
        } else {
            put(p.out[0], [&](int i) { return __uint_as_float(r[i]); });
        }
    };
    // Token i's results of a whole tile, four rows to a lane
    [[maybe_unused]] auto whole_row = [&](int tile, int i, const float (&v)[4], const float (&v1)[4]) {
        const int row = tile * p.rows + 4 * lane, there = min(p.rows - 4 * lane, p.N - row);
        if constexpr (E == DenseEnd::ENTROPY) {
            float ref, sum;
            one_token(v, there, ref, sum);
#pragma unroll
            for (int k = 0; k < SLOTS; ++k) {
                if (i >> 4 != k) continue;   // (the same for all lanes)
                const int at = __shfl_sync(0xffffffffu, target[k], 2 * (i & 15)) - row;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (at == j && j < there) p.target_logit[i] = v[j];
                if (lane / 2 == (i & 15)) dense_merge(run_ref[k], run_sum[k], ref, sum);
            }
        } else {
            auto put = [&](const DenseOut& o, const float (&x)[4]) {
                __nv_bfloat16* to = static_cast<__nv_bfloat16*>(o.p) + i * o.ld + row;
                if (there >= 4 && reinterpret_cast<uintptr_t>(to) % 8 == 0) {
                    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < there) to[j] = __float2bfloat16_rn(x[j]);
                }
            };
            if constexpr (E == DenseEnd::GATE) {
                dense_with_act(p.act, [&](auto act) {
                    float unused, h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[j] = dense_act<decltype(act)::value, false>(v[j], unused) * v1[j];
                    put(p.out[0], h);
                });
                if (p.out[1].p) {
                    put(p.out[1], v);
                    put(p.out[2], v1);
                }
            } else {
                put(p.out[0], v);
            }
        }
    };

    if (warp == 0) {
        uint32_t s = 0, ph = 0;
        int there = ahead;
        bool ok = true;
        for (int u = u0; ok && u < p.tiles; u += ustep) {
            for (int kb = lo; kb < hi; ++kb) {
                if (!wait(empty0 + 8 * s, ph ^ 1u, DEV_TIMEOUT_PRODUCER)) {
                    ok = false;
                    break;
                }
                if (there > 0)
                    --there;
                else
                    load_weights(s, kb, u);
                ptx::tma_load_2d_elected(ptx::smem_u32(smem) + s * C::STAGE_BYTES + C::MATS * C::A_BYTES, &tmX, full0 + 8 * s,
                                         kb * 64, 0);
                if (++s == C::STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) spin_ns(200000);   // copies issued before the abort land within microseconds
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t IDESC = ptx::make_idesc(1, 1, 0, 0, 128, BQ);
        constexpr uint64_t STEP = C::STAGE_BYTES / 16;
        const uint32_t stage0 = ptx::smem_u32(smem);
        const uint64_t adesc0 = ptx::sdesc_sw128(stage0, 16, 1024);
        const uint64_t qdesc0 = ptx::sdesc_sw128(stage0 + C::MATS * C::A_BYTES, 16, 1024);
        uint32_t s = 0, ph = 0;
        bool ok = true;
        for (int u = u0, j = 0; ok && u < p.tiles; u += ustep, ++j) {
            const uint32_t b = j & 1;
            if (!wait(acce0 + 8 * b, ((j >> 1) & 1) ^ 1u, DEV_TIMEOUT_MMA_ACC)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            for (int kb = lo; kb < hi; ++kb) {
                if (!wait(full0 + 8 * s, ph, DEV_TIMEOUT_MMA_FULL)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint64_t qd = qdesc0 + s * STEP;
#pragma unroll
                for (int m = 0; m < C::MATS; ++m) {
                    const uint64_t ad = adesc0 + s * STEP + m * (C::A_BYTES / 16);
                    ptx::mma_f16_x4_elected(tmem_base + b * C::COLS + (m + (kb - lo) % C::CHAINS) * BQ, ad, qd, ad + 2, qd + 2,
                                            ad + 4, qd + 4, ad + 6, qd + 6, IDESC, kb - lo >= C::CHAINS ? 1u : 0u);
                }
                ptx::mma_commit_elected(empty0 + 8 * s);
                if (++s == C::STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (ok) ptx::mma_commit_elected(accf0 + 8 * b);
        }
        if (!ok) {
            ptx::mma_commit_elected(drain_bar);
            if (lane == 0) wait_drain(drain_bar, 0, p.timeout_ns);
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3;
        for (int u = u0, j = 0; u < p.tiles; u += ustep, ++j) {
            const uint32_t b = j & 1;
            if (!wait(accf0 + 8 * b, (j >> 1) & 1, DEV_TIMEOUT_EPILOGUE)) break;
            ptx::tc_fence_after();
            const uint32_t t = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + b * C::COLS;
            // (the ring is free: a shared tile is this CTA's only one, and all its MMAs are done)
            float* sums = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
            auto release = [&]() {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_relaxed(acce0 + 8 * b);
            };
            auto columns = [&](uint32_t at, uint32_t (&r)[16]) {   // 16 of them, the chains added
                ptx::tmem_ld_32x32b_x16(at, r);
                ptx::tmem_ld_wait(r);
#pragma unroll
                for (int j = 1; j < C::CHAINS; ++j) {
                    if (j >= hi - lo) break;   // (fewer k-blocks than chains)
                    uint32_t q[16];
                    ptx::tmem_ld_32x32b_x16(at + j * BQ, q);
                    ptx::tmem_ld_wait(q);
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) + __uint_as_float(q[i]));
                }
            };
            if (E == DenseEnd::ENTROPY && share == 1) {
                dense_each<BQ / 16>([&](auto k) {
                    uint32_t r[16];
                    columns(t + 16 * decltype(k)::value, r);
                    if (decltype(k)::value == BQ / 16 - 1) release();
                    if constexpr (E == DenseEnd::ENTROPY) sixteen(u, k, r);
                });
                continue;
            }
#pragma unroll 1
            for (int c = 0; c < BQ; c += 16) {
                uint32_t r[16], r1[16];
                columns(t + c, r);
                if constexpr (C::MATS == 2) columns(t + BQ + c, r1);
                if (c + 16 == BQ) release();
                if (share > 1) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        sums[(c + i) * 128] = __uint_as_float(r[i]);
                        if constexpr (C::MATS == 2) sums[(BQ + c + i) * 128] = __uint_as_float(r1[i]);
                    }
                } else if constexpr (E != DenseEnd::ENTROPY) {
                    if (c < p.T) column(u, c, r, r1);
                }
            }
            __syncwarp();
        }
    }

    // ------------------------------------------------ shared tiles: the parts' sums, in their order
    if (share > 1) {
        __syncwarp();
        ptx::cluster_sync();   // every part's sums are in its shared memory
        if (warp >= 2 && u0 < p.tiles) {
            // a warp a token: all parts' sums of four rows a lane are on their way together
            const uint32_t sums = ptx::smem_u32(smem) + 16 * lane;
            for (int i = part + share * (warp - 2); i < p.T; i += 4 * share) {
                uint4 x[C::MATS][8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if (r >= share) continue;
                    const uint32_t at = ptx::mapa_shared(sums, static_cast<uint32_t>(r));
#pragma unroll
                    for (int m = 0; m < C::MATS; ++m) x[m][r] = ptx::ld_cluster_v4(at + 512 * (m * BQ + i));
                }
                float v[2][4] = {};
#pragma unroll
                for (int m = 0; m < C::MATS; ++m) {
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        if (r >= share) continue;
                        v[m][0] += __uint_as_float(x[m][r].x);
                        v[m][1] += __uint_as_float(x[m][r].y);
                        v[m][2] += __uint_as_float(x[m][r].z);
                        v[m][3] += __uint_as_float(x[m][r].w);
                    }
                }
                whole_row(u0, i, v[0], v[1]);
            }
        }
        __syncwarp();
        ptx::cluster_sync();   // no part leaves while another may still read its sums
    }

    if (E == DenseEnd::ENTROPY && warp >= 2 && lane % 2 == 0) {
#pragma unroll
        for (int k = 0; k < SLOTS; ++k)
            if (16 * k + lane / 2 < p.T)
                p.parts[static_cast<long long>(blockIdx.x * 4 + (warp & 3)) * p.T + 16 * k + lane / 2] =
                    make_float2(run_ref[k], run_sum[k]);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace tcl
