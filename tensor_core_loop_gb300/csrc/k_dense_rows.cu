// The passes around the dense products: operands brought onto the tensor copies' grid, the sums of
// K ranges joined, and the rows of the cross entropy.
#include "dense_launch.cuh"

namespace tcl {
namespace {

// ------------------------------------------------------------------ operands onto the grid
// A thread builds one 16-byte piece from eight elements at any address, which it reads as 4-byte words (the first
// of them may hold an element before the piece, the last one after it); a row's last pieces go
// element by element, filled up with zeros.
__global__ void dense_copy_kernel(const DenseCopies a) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const DenseCopy& c = a.job[blockIdx.y];
    const int pieces = (c.cols + 7) / 8;
    const long long n = static_cast<long long>(c.rows) * pieces, step = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
        const long long row = i / pieces;
        const int col = static_cast<int>(i - row * pieces) * 8;
        const unsigned short* from = reinterpret_cast<const unsigned short*>(c.from) + row * c.ld + col;
        uint4* to = reinterpret_cast<uint4*>(c.to + row * c.ld_to + col);
        if (col + 10 <= c.cols) {   // five aligned words hold the eight elements
            const uintptr_t at = reinterpret_cast<uintptr_t>(from);
            const uint32_t* word = reinterpret_cast<const uint32_t*>(at & ~uintptr_t(3));
            const uint32_t shift = at & 2 ? 16 : 0;
            uint32_t w[5];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = word[k];
            w[4] = shift ? word[4] : 0u;
            *to = make_uint4(__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift),
                             __funnelshift_r(w[2], w[3], shift), __funnelshift_r(w[3], w[4], shift));
        } else {
            unsigned short v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = col + k < c.cols ? from[k] : static_cast<unsigned short>(0);
            *to = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
        }
    }
}

// ------------------------------------------------------------------ K ranges joined
__global__ void dense_join_kernel(const DenseJoin a) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int quads = (a.cols + 3) / 4;
    const long long n = static_cast<long long>(a.rows) * quads, step = static_cast<long long>(gridDim.x) * blockDim.x;
    const bool vec = reinterpret_cast<uintptr_t>(a.out) % (a.f32 ? 16 : 8) == 0 && a.ld_out % 4 == 0;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
        const long long row = i / quads;
        const int col = static_cast<int>(i - row * quads) * 4;
        const float* from = a.parts + row * a.ld + col;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int z = 0; z < a.splits; ++z) {
            const float4 v = *reinterpret_cast<const float4*>(from + z * a.part);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        if (a.factor) {
            const float f = a.factor[row];
            s = f == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(s.x * f, s.y * f, s.z * f, s.w * f);
        }
        if (a.plus) {
            const float4 v = *reinterpret_cast<const float4*>(a.plus + row * a.ld_plus + col);
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        const float e[4] = {s.x, s.y, s.z, s.w};
        const long long at = row * a.ld_out + col;
        if (a.f32) {
            float* to = static_cast<float*>(a.out) + at;
            if (vec && col + 4 <= a.cols) {
                *reinterpret_cast<float4*>(to) = s;
            } else {
                for (int k = 0; k < 4 && col + k < a.cols; ++k) to[k] = e[k];
            }
        } else {
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + at;
            if (vec && col + 4 <= a.cols) {
                *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
            } else {
                for (int k = 0; k < 4 && col + k < a.cols; ++k) to[k] = __float2bfloat16_rn(e[k]);
            }
        }
    }
}

// ------------------------------------------------------------------ rows of the cross entropy
// Row t's logits l[v] left chunk sums s_i of 2^(l log2 e - ref_i). With c the largest ref_i of a
// chunk that has a sum, S = sum_i s_i 2^(ref_i - c):
//   lse = c ln 2 + ln S,  loss = lse - l[target]
// and in training, with the exponentials e[v] = 2^(l[v] log2 e - ref_i) in bf16,
//   d loss / d l[v] = e[v] 2^(ref_i - c) / S - [v = target]
// The factor grad/S of a row goes into the rows of x for the product with e^T, and into the end of
// the product e·W; the one at the target, e - S = S (exp(l[target] - lse) - 1), is worked out in
// fp32, so that a row that is nearly certain of its target keeps the small difference, and replaces
// e there. Chunks relative to another power of two (a row's chunks differ only where logits leave
// +-44 or so) are brought to c in place.
//
// The target's logit is worked out once more, as an fp32 sum on the CUDA cores: the tensor core truncates
// its sums (with K = 4096 a logit of 12 is off by 2e-5, all of a loss' error), and S gets
// the difference that makes for the target's exponential, so that a loss near zero stays one
// (16 tokens, hidden 4096: loss off by 2.8e-6 of its norm without, 2e-7 so).
// The other words' logits are off likewise, by about as much of themselves. Where all of a row are far from
// zero, most of the difference is everyone's, and moves lse instead of the target against the rest. (Hidden
// 4096, 300 tokens over 32000 words, losses of 5, root mean square of the errors in 1e-6, one channel bringing all
// logits to a level of 0 / 10 / -30 / -100: 8 / 84 / 170 / 650 with the whole difference on the target, 18 / 20 / 13 / 67
// without a second sum, 5 / 18 / 13 / 66 so; with all logits summed in fp32 4 / 16 / 29 / 130. A dropped token's lse
// stays as it is.)
//
// A block of 256 threads takes ROWS rows: eight where there are thousands of them (64 bytes of a chunk's
// row at a time), one where that leaves too few blocks.
constexpr int kRowThreads = 256;

template <int ROWS>
__global__ void __launch_bounds__(kRowThreads) entropy_rows_kernel(const EntropyRows a) {
    constexpr int KT = kRowThreads / ROWS;   // threads of a row's sums
    __shared__ float2 sh[KT][ROWS + 1];
    __shared__ float factor[ROWS], dots[kRowThreads / 32];
    auto target_of = [&](long long t) -> long long {
        if (t >= a.rows) return -1;
        const long long v = a.wide_targets ? __ldcg(static_cast<const long long*>(a.targets) + t)
                                           : __ldcg(static_cast<const int*>(a.targets) + t);
        return v < a.vocab ? v : -1;
    };
    // the rows of x: a warp each, or the block its one
    constexpr int XT = ROWS == 1 ? kRowThreads : 32;
    const int mine_of = threadIdx.x / XT, lane = threadIdx.x % XT;
    const long long mine = static_cast<long long>(blockIdx.x) * ROWS + mine_of;
    const __nv_bfloat16* x = a.x + mine * a.ld_x;
    const int pieces = a.hidden / 8, rest = pieces * 8 + lane;   // (a row may end with the buffer)
    float dot = 0.0f;
    if (const long long t = target_of(mine); t >= 0) {
        const __nv_bfloat16* w = a.w + t * a.ld_w;
#pragma unroll 4
        for (int i = lane; i < pieces; i += XT) {
            const uint4 p = __ldcg(reinterpret_cast<const uint4*>(x) + i), q = __ldcg(reinterpret_cast<const uint4*>(w) + i);
            const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dot = fmaf(__uint_as_float(u[j] << 16), __uint_as_float(v[j] << 16), dot);
                dot = fmaf(__uint_as_float(u[j] & 0xffff0000u), __uint_as_float(v[j] & 0xffff0000u), dot);
            }
        }
        auto one = [](const __nv_bfloat16* p) {
            return __uint_as_float(static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short*>(p))) << 16);
        };
        if (rest < a.hidden) dot = fmaf(one(x + rest), one(w + rest), dot);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (threadIdx.x % 32 == 0) dots[threadIdx.x / 32] = dot;
    // (The kernel before this one in the stream is the logits' own: it writes none of what is read above, and
    // what came before it had ended when it started to read. Read from the L2: what a first-level cache holds
    // may be older until the wait.)
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const int r = threadIdx.x % ROWS, k = threadIdx.x / ROWS;   // the sums: neighbouring threads, neighbouring rows
    const long long row = static_cast<long long>(blockIdx.x) * ROWS + r;
    const bool in = row < a.rows;
    const long long target = target_of(row);
    const bool kept = target >= 0;
    float logit = 0.0f, weight = 0.0f;
    if (in) {
        logit = a.target_logit[row];
        if (a.grad) weight = a.grad[row];
    }
    float c = 0.0f, s = 0.0f;
    bool other = false;   // a chunk of this thread's is relative to something else than 1
    if (in) {
#pragma unroll 8
        for (int i = k; i < a.chunks; i += KT) {
            const float2 p = a.parts[static_cast<long long>(i) * a.rows + row];
            other |= p.x != 0.0f;
            dense_merge(c, s, p.x, p.y);
        }
    }
    sh[k][r] = make_float2(c, s);
    __syncthreads();
    if (KT > 32 && k < 32) {   // (in a fixed order)
        for (int i = k + 32; i < KT; i += 32) dense_merge(c, s, sh[i][r].x, sh[i][r].y);
        sh[k][r] = make_float2(c, s);
    }
    if (KT > 32) __syncthreads();
    c = s = 0.0f;
    for (int i = 0; i < (KT < 32 ? KT : 32); ++i) dense_merge(c, s, sh[i][r].x, sh[i][r].y);
    float shift = 0.0f;
    if (kept) {
        float exact = dots[r];
        if (ROWS == 1) {
#pragma unroll
            for (int i = 1; i < kRowThreads / 32; ++i) exact += dots[i];
        }
        // Off by as much as the rest are, that is by so much of it as their mean logit is of the target's: lse takes
        // that up, and only what is left sets the target apart from the exponentials that there are. (Their mean: as
        // if words were spread normally.) Not where the sum is infinite, nor where the two differ by more than one: one of
        // them is infinite, or logits are beyond 10^5 or so; from 16 on S less what the target loses would be zero or
        // below.
        const float off = exact - logit, own = exp2f(fmaf(logit, 1.4426950408889634f, -c));
        const float mean = fmaf(c, 0.69314718055994531f, logf(fmaxf(s - own, 0.0f))) - logf(static_cast<float>(a.vocab));
        const float all = off * fminf(fmaxf(mean / logit, 0.0f), 1.0f);
        const float more = own * expm1f(off - all);
        if (fabsf(off) <= 1.0f && fabsf(more) < __int_as_float(0x7f800000)) {
            s += more;
            shift = all;
            logit = exact;
        }
    }
    const float lse = fmaf(c, 0.69314718055994531f, logf(s)) + shift;
    if (in && k == 0) {
        a.loss[row] = kept ? lse - logit : 0.0f;
        a.lse[row] = lse;
    }
    if (!a.grad) return;   // (the same for all threads)

    if (kept && (other || c != 0.0f)) {
        for (int i = k; i < a.chunks; i += KT) {
            const float ref = a.parts[static_cast<long long>(i) * a.rows + row].x;
            if (ref == c) continue;
            const float f = exp2f(ref - c);   // (a power of two: nothing is rounded again but what falls below 2^-126)
            for (int v = i * a.chunk; v < min(i * a.chunk + a.chunk, a.vocab); ++v) {
                __nv_bfloat16* e = a.e + row * a.ld_e + v;
                *e = __float2bfloat16_rn(__bfloat162float(*e) * f);
            }
        }
    }
    if (k == 0) {
        // (an infinite sum, of an infinite logit, must not pass for a token without weight)
        const float f = kept ? s < __int_as_float(0x7f800000) ? weight / s : __int_as_float(0x7fffffff) : 0.0f;
        factor[r] = f;
        if (in) a.factor[row] = f;
    }
    __syncthreads();
    if (kept && k == 0) a.e[row * a.ld_e + target] = __float2bfloat16_rn(expm1f(logit - lse) * s);
    if (mine >= a.rows) return;
    const float f = factor[mine_of];
    uint4* to = reinterpret_cast<uint4*>(a.scaled + mine * a.ld_scaled);
    auto scale = [f](uint32_t w) {   // (a dropped token's row may hold anything)
        return f == 0.0f ? 0u : pack_bf16(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
    };
#pragma unroll 4
    for (int i = lane; i < pieces; i += XT) {
        const uint4 v = reinterpret_cast<const uint4*>(x)[i];
        to[i] = make_uint4(scale(v.x), scale(v.y), scale(v.z), scale(v.w));
    }
    if (rest < a.hidden)
        a.scaled[mine * a.ld_scaled + rest] = __float2bfloat16_rn(f == 0.0f ? 0.0f : __bfloat162float(x[rest]) * f);
}

int blocks_for(long long n, int per) {
    const long long b = (n + per - 1) / per;
    return static_cast<int>(b < 1 ? 1 : b > 152 * 16 ? 152 * 16 : b);
}

}  // namespace

cudaError_t launch_dense_copies(const DenseCopies& a, cudaStream_t stream) {
    long long most = 0;
    for (int i = 0; i < a.n; ++i) {
        const long long n = static_cast<long long>(a.job[i].rows) * ((a.job[i].cols + 7) / 8);
        if (n > most) most = n;
    }
    return launch_pdl(dense_copy_kernel, dim3(blocks_for(most, 256), a.n), 256, 0, stream, a);
}

cudaError_t launch_dense_join(const DenseJoin& a, cudaStream_t stream) {
    return launch_pdl(dense_join_kernel, dim3(blocks_for(static_cast<long long>(a.rows) * ((a.cols + 3) / 4), 256)), 256, 0,
                      stream, a);
}

cudaError_t launch_entropy_rows(const EntropyRows& a, cudaStream_t stream) {
    if (a.rows > 2048) return launch_pdl(entropy_rows_kernel<8>, dim3((a.rows + 7) / 8), kRowThreads, 0, stream, a);
    return launch_pdl(entropy_rows_kernel<1>, dim3(a.rows), kRowThreads, 0, stream, a);
}

}  // namespace tcl
