// C ABI of the gated feed-forward block, of the cross entropy over a vocabulary and of the
// gradients' norm and clipping (declared in include/tcl_dense.h): argument checks, the workspace's
// layout, the choice of kernels, and the launches.
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

#include "clip_launch.cuh"
#include "dense_launch.cuh"
#include "tcl_dense.h"

namespace tcl {
namespace {

typedef __nv_bfloat16 bf16;

constexpr unsigned long long kTimeoutNs = 1000000000ull;   // bound on every in-kernel wait: 1 s
constexpr int kMostSize = 0x7ffeffff;                       // sizes are rounded up to whole tiles in 32 bits
constexpr long long kExpBytes = 1ll << 31;                  // exponentials kept at a time
// A sum's terms: the warps that wait for a tile's whole sum (dX: over two pairs) would give up after kTimeoutNs.
// 2^26 terms are 2^20 k-blocks of 0.3 us, 0.7 us where all of the operands come from HBM.
constexpr int kMostTerms = 1 << 25;

bool width(int n) { return n >= 1 && n <= kMostSize; }
bool on(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
long long up(long long x, long long m) { return (x + m - 1) / m * m; }
int tiles_of(int n, int tile) { return static_cast<int>((static_cast<long long>(n) + tile - 1) / tile); }
long long blocks64(long long k) { return (k + 63) / 64; }
// Whether the tiles of an M × N result, the narrow ones, can be counted in 32 bits.
bool countable(int M, int N) { return static_cast<long long>(tiles_of(M, 256)) * tiles_of(N, 128) <= 0x3fffffffll; }

int status_of(cudaError_t err) {
    if (err == cudaSuccess) return TCL_OK;
    cudaGetLastError();
    return err == cudaErrorInvalidValue ? TCL_ERR_DIMS : TCL_ERR_LAUNCH;
}

// A stored matrix: rows of cols values.
struct Mat {
    const bf16* p;
    long long ld;
    int rows, cols;
    bool whole = false;   // a buffer of this library's own: chunks of 64 columns are whole
    bool chunks() const { return whole || cols % 64 == 0; }
    bool copy() const { return !on(p, 16) || (rows > 1 && ld % 8); }
};

// Rows of this library's own buffers start on whole lines of 128 bytes: a box of a tensor copy whose rows
// straddle two lines each costs the L2 twice the requests (logits of 1023 tokens, hidden
// 1030, at a pitch of 1032: a k-block every 665 cycles instead of 512).
long long pitch_of(int cols) { return up(cols, 64); }

// The workspace, dealt out in 256-byte steps. Planning goes past its end; nothing is launched then.
struct Room {
    uint8_t* base;
    size_t have, used = 0;
    DenseCopies copies = {};
    template <typename T>
    T* take(long long n) {
        T* p = reinterpret_cast<T*>(base + used);
        used += static_cast<size_t>(up(n * static_cast<long long>(sizeof(T)), 256));
        return p;
    }
    // An operand as the tensor copies can read it.
    Mat operand(const void* p, long long ld, int rows, int cols) {
        Mat m = {static_cast<const bf16*>(p), rows > 1 ? ld : up(cols, 8), rows, cols};
        if (!m.copy()) return m;
        const long long pitch = pitch_of(cols);
        bf16* to = take<bf16>(pitch * rows);
        copies.job[copies.n++] = {m.p, ld, rows, cols, to, pitch};
        return {to, pitch, rows, cols, true};
    }
};

int enough(const Room& room, size_t* workspace_bytes) {
    if (room.used <= room.have) return TCL_OK;
    *workspace_bytes = room.used;
    return TCL_ERR_WORKSPACE;
}

struct Gpu {
    int sms;
    unsigned int* status;
    cudaStream_t stream;
};

int gpu_of(cudaStream_t stream, Gpu* g) {
    int dev;
    g->stream = stream;
    return device_context(&dev, &g->sms, &g->status);
}

// D = A·B^T over one operand pair or two; `mn`: the operand's rows (not K) are contiguous in memory.
struct Product {
    Mat a, b, a1, b1;
    bool a_mn, b_mn, two;
    int M, N, f32;
    void* out;
    long long ldo;
    const float* factor;
    const float* plus;
    long long ld_plus;
    int splits;
    float* parts;
};

long long k_of(const Mat& m, bool mn) { return mn ? m.rows : m.cols; }
long long blocks_of(const Product& q) {
    return blocks64(k_of(q.a, q.a_mn)) + (q.two ? blocks64(k_of(q.a1, q.a_mn)) : 0);
}

// A result of the caller's.
DenseOut result(void* p, long long ld, int cols, int rows, int f32) {
    return {p, ld, cols, on(p, 16) && (rows == 1 || ld * (f32 ? 4 : 2) % 16 == 0)};
}

// What a launch costs, in microseconds, measured on a GB300: a k-block of a tile, a tile's end (where it does
// not hide behind the next tile's k-blocks), a launch, and the joining of K ranges.
// (The way from the L2 bounds all but wide tiles with K contiguous in A: a narrow tile has 2/3 of a wide one's operand
// bytes and half of its MMAs, and boxes of contiguous rows come in at two thirds of the rate of boxes of K.)
double block_us(int bn, bool mn = false) { return mn ? (bn == 256 ? 0.32 : 0.30) : bn == 256 ? 0.27 : 0.22; }
double tile_us(int bn) { return bn == 256 ? 3.0 : 2.0; }
// The least time between a pair's tiles: what their epilogue warps and the memory take for one (rows off the 16-byte
// grid are stored by the warps themselves).
double end_us(int bn, int f32, bool by_copy) { return (bn == 256 ? 0.9 : 0.5) * (f32 ? 1.6 : 1.0) * (by_copy ? 1.0 : 2.2); }
constexpr double kLaunchUs = 5.0;

// A launch of up to kDenseProblems products: the tiles' width, K ranges of the first one (the longest),
// and its units' way to the pairs of SMs (dense_walk).
struct Group {
    Product* q;
    int n, bn;
    int units, long_units, extra, pairs;
    bool deep;   // six k-blocks and a slab
};

// Deals the units out; the time that takes.
double deal(Group& g, int sms) {
    long long units = 0, first = 0;
    double each[2] = {0.0, 0.0}, work = 0.0;   // a unit of the first product, the longest of the others
    double two_slabs = 0.0, one_slab = 0.0, last = 0.0;
    for (int i = 0; i < g.n; ++i) {
        const Product& q = g.q[i];
        const long long n = static_cast<long long>(tiles_of(q.M, 256)) * tiles_of(q.N, g.bn) * q.splits;
        const bool parts = q.splits > 1;
        const double loop = block_us(g.bn, q.a_mn) * std::ceil(static_cast<double>(blocks_of(q)) / q.splits) + 0.3;
        const double end = end_us(g.bn, parts || q.f32, parts || result(q.out, q.ldo, q.N, q.M, q.f32).tma);
        const double us = std::max(loop, end);
        two_slabs += us * static_cast<double>(n);
        one_slab += std::max(0.97 * loop, 1.4 * end) * static_cast<double>(n);
        last = std::max(last, end);
        units += n;
        work += us * static_cast<double>(n);
        if (i == 0) first = n;
        each[i > 0] = std::max(each[i > 0], us);
    }
    g.units = static_cast<int>(std::min(units, 0x40000000ll));
    g.pairs = static_cast<int>(std::min<long long>(sms / 2, units));
    g.deep = one_slab + 0.25 * last * g.pairs < two_slabs;   // (each pair's last end shows)
    g.long_units = static_cast<int>(std::min(first, 0x40000000ll));
    const int r0 = g.long_units % g.pairs;
    g.extra = g.n > 1 && r0 ? static_cast<int>(each[0] / each[1] + 0.5) : 0;
    // the pair that ends last: of those with one more of the long units, or of the others
    const long long rest = units - first, late = static_cast<long long>(g.extra) * (g.pairs - r0);
    const long long rounds = rest > late ? (rest - late + g.pairs - 1) / g.pairs : 0;
    const double most = each[0] * static_cast<double>(first / g.pairs + (r0 > 0)) + each[1] * static_cast<double>(rounds);
    const double others = each[0] * static_cast<double>(first / g.pairs) +
                          each[1] * static_cast<double>(rounds + std::min<long long>(g.extra, (rest + g.pairs - r0 - 1) / (g.pairs - r0)));
    return std::max(std::max(most, r0 < g.pairs ? others : 0.0), work / g.pairs) + tile_us(g.bn) + kLaunchUs;
}

// Chooses width and K ranges by the costs above; the time.
double choose(Group& g, int sms) {
    double least = 0.0;
    int bn = 0, splits = 1;
    const long long kb = blocks_of(g.q[0]);
    for (int i = 1; i < g.n; ++i) g.q[i].splits = 1;
    static constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
    for (g.bn = 256; g.bn >= 128; g.bn /= 2) {
        const long long tiles = static_cast<long long>(tiles_of(g.q[0].M, 256)) * tiles_of(g.q[0].N, g.bn);
        for (const int s : kSplits) {
            if (s > 1 && (s * 4 > kb || tiles * s > 2 * sms)) break;   // (short ranges; more units than hide their ends)
            g.q[0].splits = s;
            double us = deal(g, sms);
            // the ranges' sums are written and read again, at 5 TB/s
            if (s > 1) us += kLaunchUs + 8.0 * s * g.q[0].M * static_cast<double>(g.q[0].N) / 5e6;
            if (!bn || us < 0.98 * least) {
                bn = g.bn;
                splits = s;
                least = us;
            }
        }
    }
    g.bn = bn;
    g.q[0].splits = splits;
    deal(g, sms);
    return least;
}

// Room for the sums of K ranges.
void reserve(Room& room, Group& g) {
    for (int i = 0; i < g.n; ++i) {
        Product& q = g.q[i];
        q.parts = q.splits > 1 ? room.take<float>(static_cast<long long>(q.splits) * q.M * up(q.N, 4)) : nullptr;
    }
}

// Boxes of 64 columns × `rows` rows of a K-contiguous operand; of 64 rows × `rows` columns of the other
// kind (two copies of 64 columns where the matrix has no whole chunks of them).
int map_of(const Mat& m, bool mn, int rows, CUtensorMap* out, bool chunks = false) {
    if (mn && chunks)
        return tensor_map_bf16_chunks(m.p, blocks64(m.cols), m.rows, m.ld * 2, 64, rows / 64, out);
    return tensor_map_bf16(m.p, m.cols, m.rows, m.ld * 2, mn ? 64 : rows, out);
}

int map_out(const DenseOut& o, int f32, int rows, int mats, CUtensorMap* out) {
    if (!o.tma) return TCL_OK;
    const long long row = up(o.ld * (f32 ? 4 : 2), 16);   // (a single row never steps to a second one)
    return tensor_map_result(o.p, !f32, o.cols, rows, mats, row, row * rows, out);
}

int launch_pairs(DenseLaunch& l, const Gpu& g) {
    l.p.timeout_ns = kTimeoutNs;
    l.p.status = g.status;
    l.stream = g.stream;
    if (l.p.units > 0x3fffffff) return TCL_ERR_DIMS;
    return status_of(launch_dense_pair(l));
}

int run(const Group& g, const Gpu& gpu) {
    DenseLaunch l = {};
    l.end = DenseEnd::STORE;
    l.bn = g.bn;
    l.pairs = g.pairs;
    DenseParams& p = l.p;
    p.n = g.n;
    p.units = g.units;
    p.long_units = g.long_units;
    p.extra = g.extra;
    p.deep = g.deep;
    int st, first = 0;
    for (int i = 0; i < g.n; ++i) {
        const Product& q = g.q[i];
        DenseProblem& d = p.q[i];
        d.a_3d = q.a.chunks() && (!q.two || q.a1.chunks());
        d.b_3d = q.b.chunks() && (!q.two || q.b1.chunks());
        const int br = g.bn / 2;
        if ((st = map_of(q.a, q.a_mn, 128, &l.maps.a[i][0], d.a_3d)) || (st = map_of(q.b, q.b_mn, br, &l.maps.b[i][0], d.b_3d)))
            return st;
        if (q.two && ((st = map_of(q.a1, q.a_mn, 128, &l.maps.a[i][1], d.a_3d)) ||
                      (st = map_of(q.b1, q.b_mn, br, &l.maps.b[i][1], d.b_3d))))
            return st;
        d.M = q.M;
        d.N = q.N;
        d.kb0 = static_cast<int>(blocks64(k_of(q.a, q.a_mn)));
        d.kb1 = static_cast<int>(blocks_of(q)) - d.kb0;
        d.tiles_m = tiles_of(q.M, 256);
        d.tiles_n = tiles_of(q.N, g.bn);
        d.splits = q.splits;
        d.first = first;
        d.a_mn = q.a_mn;
        d.b_mn = q.b_mn;
        const long long pitch = up(q.N, 4);
        if (q.splits > 1) {
            d.f32 = 1;
            d.out = {q.parts, pitch, static_cast<int>(pitch), 1};
        } else {
            d.f32 = q.f32;
            d.out = result(q.out, q.ldo, q.N, q.M, q.f32);
            d.factor = q.factor;
            d.plus = q.plus;
            d.ld_plus = q.ld_plus;
        }
        if ((st = map_out(d.out, d.f32, q.M, q.splits, &l.maps.c[i]))) return st;
        if (g.units < 0x40000000) first += d.tiles_m * d.tiles_n * d.splits;
    }
    if ((st = launch_pairs(l, gpu))) return st;
    for (int i = 0; i < g.n; ++i) {
        const Product& q = g.q[i];
        const long long pitch = up(q.N, 4);
        if (q.splits > 1 && (st = status_of(launch_dense_join({q.parts, pitch, pitch * q.M, q.splits, q.M, q.N, q.f32, q.factor,
                                                               q.plus, q.ld_plus, q.out, q.ldo},
                                                              gpu.stream))))
            return st;
    }
    return TCL_OK;
}

// A long product (q[0]) and those that do not depend on it (q[1 ..n)): one launch, or two where the first
// keeps the GPU busy for two rounds of tiles by itself. (Pairs that work on different products do not
// walk K together, so that less of what they read is in the L2: gradients of 8192 tokens,
// hidden 4096, vocabulary 131072 in one launch 3.6 % slower than in two; those of 1023 tokens,
// hidden 1030, vocabulary 32001 5 % faster.)
struct Launches {
    Group g[2];
    int n;
};

Launches arrange(Product* q, int n, int sms) {
    Launches l;
    const long long tiles = static_cast<long long>(tiles_of(q[0].M, 256)) * tiles_of(q[0].N, 256);
    l.n = tiles >= sms ? 2 : 1;
    l.g[0] = {q, l.n == 2 ? 1 : n};
    l.g[1] = {q + 1, n - 1};
    for (int i = 0; i < l.n; ++i) choose(l.g[i], sms);
    return l;
}

void reserve(Room& room, Launches& l) {
    for (int i = 0; i < l.n; ++i) reserve(room, l.g[i]);
}

int run(const Launches& l, const Gpu& gpu) {
    int st = TCL_OK;
    for (int i = 0; i < l.n && !st; ++i) st = run(l.g[i], gpu);
    return st;
}

// The launch of one M × N result with an end of its own, K contiguous in A.
DenseLaunch ended(DenseEnd end, int M, int N, long long k, int cols256, const Gpu& g) {
    DenseLaunch l = {};
    l.end = end;
    // narrow tiles where wide ones leave SMs without a tile and the tiles' ends show
    const long long wide = static_cast<long long>(tiles_of(M, 256)) * tiles_of(N, cols256);
    const long long narrow = static_cast<long long>(tiles_of(M, 256)) * tiles_of(N, cols256 / 2);
    const long long pairs = g.sms / 2;
    auto us = [&](long long tiles, int bn) {
        return static_cast<double>((tiles + pairs - 1) / pairs) * (block_us(bn) * static_cast<double>(blocks64(k)) + 0.3) + tile_us(bn);
    };
    l.bn = us(narrow, 128) < us(wide, 256) ? 128 : 256;
    DenseProblem& d = l.p.q[0];
    d.M = M;
    d.N = N;
    d.kb0 = static_cast<int>(blocks64(k));
    d.tiles_m = tiles_of(M, 256);
    d.tiles_n = tiles_of(N, l.bn == 256 ? cols256 : cols256 / 2);
    d.splits = 1;
    l.p.n = 1;
    l.p.units = l.p.long_units = static_cast<int>(std::min(l.bn == 256 ? wide : narrow, 0x40000000ll));
    l.pairs = static_cast<int>(std::min<long long>(pairs, l.p.units));
    return l;
}

// ------------------------------------------------------------------ few tokens

// Whether `values` weights are read by the kernel for few tokens. Measured in CUDA graphs on a GB300, the block,
// microseconds, it against tiles on pairs of SMs:
//   hidden × inner   tokens = 1         16          64          100
//   4096 × 14336      59.4 | 99.6   60.5 | 79.5   65.6 | 82.0   71.5 | 83.9
//   4096 × 8192       40.5 | 63.8   41.1 | 51.5   46.9 | 53.1   54.4 | 53.9
//   2048 × 5632       20.5 | 35.3   20.5 | 28.7   24.7 | 28.7   30.7 | 28.7
//   512 × 1408        12.3 | 16.6   12.3 | 16.4   16.4 | 16.4   20.5 | 16.4
// (cross entropy over 131072 × 4096: 64 tokens 170 | 190, 128 tokens 185 | 193)
bool is_few(int tokens, long long values) { return tokens <= 64 || (tokens <= 128 && values > 40000000ll); }

int launch_few(DenseEnd end, const Mat& x, const Mat& w0, const Mat* w1, DenseFewParams p, const Gpu& g, int* ctas = nullptr) {
    DenseFewLaunch l = {};
    l.end = end;
    l.bq = p.T <= 16 ? 16 : p.T <= 32 ? 32 : p.T <= 64 ? 64 : 128;
    p.N = w0.rows;
    p.num_kb = static_cast<int>(blocks64(w0.cols));
    p.timeout_ns = kTimeoutNs;
    p.status = g.status;
    // Rows of a tile and CTAs that share one: the least time of the CTA with the most to load. In units of a
    // row's k-block (128 bytes): a tile's end counts as 400 of them, the exchange of a shared tile's sums as 1500.
    long long least = 0;
    for (int split = 1; split <= 8; split *= 2) {
        if (split > 1 && p.num_kb < 2 * split) break;
        const int places = dense_few_clusters(split, g.sms);
        for (int rows = 128; rows >= 64; rows -= 8) {
            const long long tiles = tiles_of(p.N, rows), waves = (tiles + places - 1) / places;
            if (split > 1 && waves > 1) continue;   // (a shared tile is its CTAs' only one)
            const long long cost = waves * (static_cast<long long>(rows) * ((p.num_kb + split - 1) / split) + 400) +
                                   (split > 1 ? 1500 : 0);
            if (least && cost >= least) continue;
            least = cost;
            p.split = split;
            p.rows = rows;
            p.tiles = static_cast<int>(tiles);
        }
    }
    int st;
    if ((st = tensor_map_bf16(x.p, x.cols, x.rows, x.ld * 2, l.bq, &l.x)) || (st = map_of(w0, false, p.rows, &l.w[0]))) return st;
    if (w1 && (st = map_of(*w1, false, p.rows, &l.w[1]))) return st;
    l.p = p;
    l.grid = std::min(p.split > 1 ? p.tiles : g.sms, p.tiles) * p.split;
    l.stream = g.stream;
    if (ctas) *ctas = l.grid;
    return status_of(launch_dense_few(l));
}

// ------------------------------------------------------------------ the feed-forward block

struct Ffn {
    int T, H, F, act;
    Mat x, wg, wu, wd;
};

int ffn_sizes(int tokens, int hidden, int inner, int act) {
    if (tokens < 0 || tokens > kMostSize || !width(hidden) || !width(inner)) return TCL_ERR_DIMS;
    if (hidden > kMostTerms || inner > kMostTerms) return TCL_ERR_DIMS;
    // (the gate's tiles are half as wide; the gradients' products share a launch)
    if (!countable(tokens, 2 * std::min(inner, 0x3fffffff)) || !countable(tokens, hidden) || !countable(inner, hidden) ||
        !countable(hidden, inner))
        return TCL_ERR_DIMS;
    return act < 0 || act > 2 ? TCL_ERR_CONFIG : TCL_OK;
}

int gate_pairs(const Ffn& f, bf16* gate, bf16* upp, bf16* h, long long ldk, const Gpu& g) {
    DenseLaunch l = ended(DenseEnd::GATE, f.T, f.F, f.H, 128, g);
    int st;
    if ((st = map_of(f.x, false, 128, &l.maps.a[0][0])) || (st = map_of(f.wg, false, l.bn / 2, &l.maps.b[0][0])) ||
        (st = map_of(f.wu, false, l.bn / 2, &l.maps.b[0][1])))
        return st;
    l.p.deep = l.p.q[0].kb0 >= 12;   // (12 k-blocks: a tile's ends, gate and up kept, do not show beside them)
    l.p.act = f.act;
    void* const to[3] = {h, gate, upp};
    for (int i = 0; i < (gate ? 3 : 1); ++i) {
        DenseOut& o = i ? l.p.more[i - 1] : l.p.q[0].out;
        o = {to[i], ldk, static_cast<int>(up(f.F, 8)), 1};
        if ((st = map_out(o, 0, f.T, 1, &l.maps.c[i]))) return st;
    }
    return launch_pairs(l, g);
}

int gate_grad(const Ffn& f, const Mat& grad, const bf16* gate, const bf16* upp, long long ldk, bf16* dg, bf16* du,
              long long ldd, const Gpu& g) {
    DenseLaunch l = ended(DenseEnd::GATE_GRAD, f.T, f.F, f.H, 256, g);
    int st;
    if ((st = map_of(grad, false, 128, &l.maps.a[0][0])) || (st = map_of(f.wd, true, l.bn / 2, &l.maps.b[0][0], f.wd.chunks()))) return st;
    l.p.q[0].b_3d = f.wd.chunks();
    // four warps end a tile in some 25,000 cycles: behind 56 k-blocks of the next tile, where there is one (4096 × 14336,
    // all gradients of 1024 tokens 402 us to 392, of 512 tokens 241 to 239; of 130, a tile a pair, 158.5 to 159.2)
    l.p.deep = l.p.q[0].kb0 >= 56 && l.p.units > l.pairs;
    l.p.act = f.act;
    for (int i = 0; i < 2; ++i)   // 64 columns × 32 rows at a time
        if ((st = tensor_map_bf16(i ? upp : gate, f.F, f.T, ldk * 2, 32, &l.maps.a[1][i]))) return st;
    l.p.q[0].out = {dg, ldd, static_cast<int>(up(f.F, 8)), 1};
    l.p.more[0] = {du, ldd, static_cast<int>(up(f.F, 8)), 1};
    if ((st = map_out(l.p.q[0].out, 0, f.T, 1, &l.maps.c[0])) || (st = map_out(l.p.more[0], 0, f.T, 1, &l.maps.c[1]))) return st;
    return launch_pairs(l, g);
}

int zeros(void* p, long long ld, int rows, int cols, int f32, cudaStream_t stream) {
    const size_t es = f32 ? 4 : 2;
    return status_of(cudaMemset2DAsync(p, ld * es, 0, cols * es, rows, stream));
}

// ------------------------------------------------------------------ the cross entropy

struct Entropy {
    int T, H, V;
    Mat x, w;
    const void* targets;
    int target_bytes;
    float *loss, *lse;
};

int entropy_checks(int tokens, int hidden, int vocab, const void* X, int ldx, const void* W, int ldw, const void* targets,
                   int target_bytes, const float* loss, const float* lse) {
    if (tokens < 0 || tokens > kMostSize || !width(hidden) || !width(vocab) || hidden > kMostTerms) return TCL_ERR_DIMS;
    if (!countable(tokens, vocab) || !countable(tokens, hidden) || !countable(vocab, hidden)) return TCL_ERR_DIMS;
    if (target_bytes != 4 && target_bytes != 8) return TCL_ERR_CONFIG;
    if (tokens && (!X || !W || !targets || !loss || !lse)) return TCL_ERR_NULL;
    if (ldx < hidden || ldw < hidden) return TCL_ERR_LD;
    if (!on(X, 2) || !on(W, 2) || !on(targets, target_bytes) || !on(loss, 4) || !on(lse, 4)) return TCL_ERR_ALIGN;
    return TCL_OK;
}

// The logits of rows [t0, t0 + rows) and what is kept of them; e NULL: sums alone. `chunk`: columns of a sum.
int entropy_pairs(const Entropy& n, int t0, int rows, bf16* e, long long lde, float2* parts, float* target_logit, int* chunk,
                  const Gpu& g) {
    DenseLaunch l = ended(DenseEnd::ENTROPY, rows, n.V, n.H, 256, g);
    const Mat x = {n.x.p + t0 * n.x.ld, n.x.ld, rows, n.H};
    int st;
    if ((st = map_of(x, false, 128, &l.maps.a[0][0])) || (st = map_of(n.w, false, l.bn / 2, &l.maps.b[0][0]))) return st;
    DenseParams& p = l.p;
    p.targets = static_cast<const uint8_t*>(n.targets) + static_cast<long long>(t0) * n.target_bytes;
    p.wide_targets = n.target_bytes == 8;
    p.parts = parts;
    p.target_logit = target_logit;
    p.exps = e != nullptr;
    p.deep = e ? 0 : 2;
    if (e) {
        p.q[0].out = {e, lde, static_cast<int>(up(n.V, 8)), 1};
        if ((st = map_out(p.q[0].out, 0, rows, 1, &l.maps.c[0]))) return st;
    }
    *chunk = l.bn / 2;
    return launch_pairs(l, g);
}

EntropyRows entropy_rows(const Entropy& n, int t0, int rows, int chunks, int chunk, const float2* parts, const float* target_logit) {
    EntropyRows r = {};
    r.parts = parts;
    r.chunks = chunks;
    r.chunk = chunk;
    r.rows = rows;
    r.vocab = n.V;
    r.target_logit = target_logit;
    r.targets = static_cast<const uint8_t*>(n.targets) + static_cast<long long>(t0) * n.target_bytes;
    r.wide_targets = n.target_bytes == 8;
    r.loss = n.loss + t0;
    r.lse = n.lse + t0;
    r.x = n.x.p + t0 * n.x.ld;
    r.ld_x = n.x.ld;
    r.w = n.w.p;
    r.ld_w = n.w.ld;
    r.hidden = n.H;
    return r;
}

// ------------------------------------------------------------------ clipping

int clip_checks(int count, const void* const* from, const long long* lengths, const int* types, const float* norm) {
    if (count < 0) return TCL_ERR_DIMS;
    if (!norm || (count && (!from || !lengths || !types))) return TCL_ERR_NULL;
    if (!on(norm, 4)) return TCL_ERR_ALIGN;
    for (int i = 0; i < count; ++i) {
        if (types[i] != TCL_OUT_F32 && types[i] != TCL_OUT_BF16) return TCL_ERR_CONFIG;
        if (lengths[i] < 0 || lengths[i] > (1ll << 48)) return TCL_ERR_DIMS;
        if (lengths[i] && !from[i]) return TCL_ERR_NULL;
        if (!on(from[i], types[i] == TCL_OUT_F32 ? 4 : 2)) return TCL_ERR_ALIGN;
    }
    return TCL_OK;
}

// Whether a result shares memory with another one, or with an operand that is not its own: the blocks of one tensor
// would read what those of the other may have scaled already.
int overlap_checks(int count, const void* const* from, void* const* to, const long long* lengths, const int* types) {
    struct Span {
        uintptr_t lo, hi;
        int i;
    };
    const std::unique_ptr<Span[]> spans(new (std::nothrow) Span[count ? count : 1]);
    if (!spans) return TCL_ERR_NO_MEMORY;
    auto span = [&](const void* p, int i) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        return Span{lo, lo + static_cast<uintptr_t>(lengths[i]) * (types[i] == TCL_OUT_F32 ? 4 : 2), i};
    };
    Span* end = spans.get();
    for (int i = 0; i < count; ++i)
        if (lengths[i]) *end++ = span(to[i], i);
    std::sort(spans.get(), end, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    for (Span* s = spans.get(); s + 1 < end; ++s)
        if (s->hi > s[1].lo) return TCL_ERR_CONFIG;
    for (int i = 0; i < count; ++i) {
        if (!lengths[i] || from[i] == to[i]) continue;   // (its own span, and no two of those overlap)
        const Span a = span(from[i], i);
        const Span* s = std::upper_bound(spans.get(), end, a.lo, [](uintptr_t lo, const Span& b) { return lo < b.hi; });
        if (s < end && s->lo < a.hi) return TCL_ERR_CONFIG;
    }
    return TCL_OK;
}

// Calls f with one launch's tensors after another's: those of one type, kClipTensors at most.
template <class F>
int each_launch(int count, const void* const* from, void* const* to, const long long* lengths, const int* types, F f) {
    long long total = 0;
    for (int i = 0; i < count; ++i) total += lengths[i];
    // pieces that give every block several, of whole steps of the kernels' loops
    const long long piece = std::min(65536ll, std::max(8192ll, total / (4 * kClipBlocks) / 8192 * 8192));
    for (int f32 = 0; f32 < 2; ++f32) {
        ClipTensors a;
        a.n = 0;
        a.f32 = f32;
        a.piece = static_cast<int>(piece);
        a.pieces = 0;
        for (int i = 0; i <= count; ++i) {
            if (a.n == kClipTensors || (i == count && a.n)) {
                if (const int st = f(a)) return st;
                a.n = 0;
                a.pieces = 0;
            }
            if (i == count || (types[i] == TCL_OUT_F32) != f32 || lengths[i] == 0) continue;
            a.t[a.n++] = {from[i], to ? to[i] : nullptr, lengths[i], a.pieces};
            a.pieces += (lengths[i] + piece - 1) / piece;
        }
    }
    return TCL_OK;
}

}  // namespace
}  // namespace tcl

using namespace tcl;

extern "C" {

int tcl_gated_ffn(int tokens, int hidden, int inner, const void* X, int ldx, const void* Wgate, int ld_gate, const void* Wup,
                  int ld_up, const void* Wdown, int ld_down, int act, void* gate, void* upp, void* h, int ld_kept, void* out,
                  int ldo, void* workspace, size_t* workspace_bytes, cudaStream_t stream) {
    if (const int st = ffn_sizes(tokens, hidden, inner, act)) return st;
    if (!workspace_bytes || (*workspace_bytes && !workspace)) return TCL_ERR_NULL;
    if (tokens && (!X || !Wgate || !Wup || !Wdown || !h || !out || !gate != !upp)) return TCL_ERR_NULL;
    if (ldx < hidden || ld_gate < hidden || ld_up < hidden || ld_down < inner || ldo < hidden || ld_kept < inner || ld_kept % 8)
        return TCL_ERR_LD;
    if (!on(X, 2) || !on(Wgate, 2) || !on(Wup, 2) || !on(Wdown, 2) || !on(out, 2) || !on(gate, 16) || !on(upp, 16) ||
        !on(h, 16) || !on(workspace, 256))
        return TCL_ERR_ALIGN;
    Gpu g;
    if (const int st = gpu_of(stream, &g)) return st;
    if (tokens == 0) return TCL_OK;
    Room room{static_cast<uint8_t*>(workspace), *workspace_bytes};
    Ffn f = {tokens, hidden, inner, act, room.operand(X, ldx, tokens, hidden), room.operand(Wgate, ld_gate, inner, hidden),
             room.operand(Wup, ld_up, inner, hidden), room.operand(Wdown, ld_down, hidden, inner)};
    const Mat kept = {static_cast<const bf16*>(h), ld_kept, tokens, inner};
    Product q = {};
    q.a = kept;
    q.b = f.wd;
    q.M = tokens;
    q.N = hidden;
    q.out = out;
    q.ldo = ldo;
    Group down = {&q, 1};
    const bool few = is_few(tokens, static_cast<long long>(hidden) * inner);
    if (!few) {
        choose(down, g.sms);
        reserve(room, down);
    }
    if (const int st = enough(room, workspace_bytes)) return st;
    const auto lock = library_lock();
    int st;
    if (room.copies.n && (st = status_of(launch_dense_copies(room.copies, stream)))) return st;
    if (!few) {
        if ((st = gate_pairs(f, static_cast<bf16*>(gate), static_cast<bf16*>(upp), static_cast<bf16*>(h), ld_kept, g))) return st;
        return run(down, g);
    }
    DenseFewParams p = {};
    p.T = tokens;
    p.act = act;
    p.out[0] = {h, ld_kept, 0, 0};
    p.out[1] = {gate, ld_kept, 0, 0};
    p.out[2] = {upp, ld_kept, 0, 0};
    if ((st = launch_few(DenseEnd::GATE, f.x, f.wg, &f.wu, p, g))) return st;
    p.out[0] = {out, ldo, 0, 0};
    p.early = 1;
    return launch_few(DenseEnd::STORE, kept, f.wd, nullptr, p, g);
}

int tcl_gated_ffn_grad(int tokens, int hidden, int inner, const void* grad, int ld_grad, const void* X, int ldx,
                       const void* Wgate, int ld_gate, const void* Wup, int ld_up, const void* Wdown, int ld_down, int act,
                       const void* gate, const void* upp, const void* h, int ld_kept, void* dX, int ld_dx, void* dWgate,
                       int ld_dgate, void* dWup, int ld_dup, void* dWdown, int ld_ddown, int w_type, void* workspace,
                       size_t* workspace_bytes, cudaStream_t stream) {
    if (const int st = ffn_sizes(tokens, hidden, inner, act)) return st;
    if (tokens > kMostTerms) return TCL_ERR_DIMS;
    if (w_type != TCL_OUT_F32 && w_type != TCL_OUT_BF16) return TCL_ERR_CONFIG;
    if (!workspace_bytes || (*workspace_bytes && !workspace) || !dWgate || !dWup || !dWdown) return TCL_ERR_NULL;
    if (tokens && (!grad || !X || !Wgate || !Wup || !Wdown || !gate || !upp || !h || !dX)) return TCL_ERR_NULL;
    if (ldx < hidden || ld_grad < hidden || ld_gate < hidden || ld_up < hidden || ld_down < inner || ld_dx < hidden ||
        ld_dgate < hidden || ld_dup < hidden || ld_ddown < inner || ld_kept < inner || ld_kept % 8)
        return TCL_ERR_LD;
    const int f32 = w_type == TCL_OUT_F32, es = f32 ? 4 : 2;
    if (!on(grad, 2) || !on(X, 2) || !on(Wgate, 2) || !on(Wup, 2) || !on(Wdown, 2) || !on(dX, 2) || !on(dWgate, es) ||
        !on(dWup, es) || !on(dWdown, es) || !on(gate, 16) || !on(upp, 16) || !on(h, 16) || !on(workspace, 256))
        return TCL_ERR_ALIGN;
    Gpu g;
    int st;
    if ((st = gpu_of(stream, &g))) return st;
    if (tokens == 0) {
        if ((st = zeros(dWgate, ld_dgate, inner, hidden, f32, stream)) || (st = zeros(dWup, ld_dup, inner, hidden, f32, stream)))
            return st;
        return zeros(dWdown, ld_ddown, hidden, inner, f32, stream);
    }
    Room room{static_cast<uint8_t*>(workspace), *workspace_bytes};
    Ffn f = {tokens, hidden, inner, act, room.operand(X, ldx, tokens, hidden), room.operand(Wgate, ld_gate, inner, hidden),
             room.operand(Wup, ld_up, inner, hidden), room.operand(Wdown, ld_down, hidden, inner)};
    const Mat gr = room.operand(grad, ld_grad, tokens, hidden);
    const Mat kept = {static_cast<const bf16*>(h), ld_kept, tokens, inner};
    const long long ldd = pitch_of(inner);
    bf16* dg = room.take<bf16>(ldd * tokens);
    bf16* du = room.take<bf16>(ldd * tokens);
    const Mat mg = {dg, ldd, tokens, inner, true}, mu = {du, ldd, tokens, inner, true};
    Product q[4] = {};
    // dX = dgate·Wgate + dup·Wup: one product over both
    q[0].a = mg;
    q[0].b = f.wg;
    q[0].a1 = mu;
    q[0].b1 = f.wu;
    q[0].two = q[0].b_mn = true;
    q[0].M = tokens;
    q[0].N = hidden;
    q[0].out = dX;
    q[0].ldo = ld_dx;
    const Mat left[3] = {mg, mu, gr}, right[3] = {f.x, f.x, kept};
    void* const to[3] = {dWgate, dWup, dWdown};
    const int ld[3] = {ld_dgate, ld_dup, ld_ddown};
    for (int i = 0; i < 3; ++i) {
        Product& w = q[i + 1];
        w.a = left[i];
        w.b = right[i];
        w.a_mn = w.b_mn = true;
        w.M = left[i].cols;
        w.N = right[i].cols;
        w.f32 = f32;
        w.out = to[i];
        w.ldo = ld[i];
    }
    Launches all = arrange(q, 4, g.sms);
    reserve(room, all);
    if ((st = enough(room, workspace_bytes))) return st;
    const auto lock = library_lock();
    if (room.copies.n && (st = status_of(launch_dense_copies(room.copies, stream)))) return st;
    if ((st = gate_grad(f, gr, static_cast<const bf16*>(gate), static_cast<const bf16*>(upp), ld_kept, dg, du, ldd, g))) return st;
    return run(all, g);
}

int tcl_cross_entropy(int tokens, int hidden, int vocab, const void* X, int ldx, const void* W, int ldw, const void* targets,
                      int target_bytes, float* loss, float* lse, void* workspace, size_t* workspace_bytes,
                      cudaStream_t stream) {
    if (const int st = entropy_checks(tokens, hidden, vocab, X, ldx, W, ldw, targets, target_bytes, loss, lse)) return st;
    if (!workspace_bytes || (*workspace_bytes && !workspace)) return TCL_ERR_NULL;
    if (!on(workspace, 256)) return TCL_ERR_ALIGN;
    Gpu g;
    int st;
    if ((st = gpu_of(stream, &g))) return st;
    if (tokens == 0) return TCL_OK;
    Room room{static_cast<uint8_t*>(workspace), *workspace_bytes};
    const Entropy n = {tokens, hidden, vocab, room.operand(X, ldx, tokens, hidden), room.operand(W, ldw, vocab, hidden), targets,
                       target_bytes, loss, lse};
    const bool few = is_few(tokens, static_cast<long long>(hidden) * vocab);
    int chunks = few ? 4 * g.sms : tiles_of(vocab, 64), chunk = 0;
    float2* parts = room.take<float2>(static_cast<long long>(chunks) * tokens);
    float* target_logit = room.take<float>(tokens);
    if ((st = enough(room, workspace_bytes))) return st;
    const auto lock = library_lock();
    if (room.copies.n && (st = status_of(launch_dense_copies(room.copies, stream)))) return st;
    if (few) {
        DenseFewParams p = {};
        p.T = tokens;
        p.targets = targets;
        p.wide_targets = target_bytes == 8;
        p.parts = parts;
        p.target_logit = target_logit;
        int ctas = 0;
        st = launch_few(DenseEnd::ENTROPY, n.x, n.w, nullptr, p, g, &ctas);
        chunks = 4 * ctas;
    } else {
        st = entropy_pairs(n, 0, tokens, nullptr, 0, parts, target_logit, &chunk, g);
        chunks = tiles_of(vocab, chunk);
    }
    if (st) return st;
    return status_of(launch_entropy_rows(entropy_rows(n, 0, tokens, chunks, chunk, parts, target_logit), stream));
}

int tcl_cross_entropy_grad(int tokens, int hidden, int vocab, const void* X, int ldx, const void* W, int ldw,
                           const void* targets, int target_bytes, const float* grad, float* loss, float* lse, void* dX,
                           int ld_dx, void* dW, int ld_dw, int w_type, void* workspace, size_t* workspace_bytes,
                           cudaStream_t stream) {
    if (const int st = entropy_checks(tokens, hidden, vocab, X, ldx, W, ldw, targets, target_bytes, loss, lse)) return st;
    if (vocab > kMostTerms) return TCL_ERR_DIMS;   // (tokens come in pieces of 2^24 at most)
    if (w_type != TCL_OUT_F32 && w_type != TCL_OUT_BF16) return TCL_ERR_CONFIG;
    if (!workspace_bytes || (*workspace_bytes && !workspace) || !dW || (tokens && (!grad || !dX))) return TCL_ERR_NULL;
    if (ld_dx < hidden || ld_dw < hidden) return TCL_ERR_LD;
    const int f32 = w_type == TCL_OUT_F32;
    if (!on(grad, 4) || !on(dX, 2) || !on(dW, f32 ? 4 : 2) || !on(workspace, 256)) return TCL_ERR_ALIGN;
    Gpu g;
    int st;
    if ((st = gpu_of(stream, &g))) return st;
    if (tokens == 0) return zeros(dW, ld_dw, vocab, hidden, f32, stream);
    Room room{static_cast<uint8_t*>(workspace), *workspace_bytes};
    const Entropy n = {tokens, hidden, vocab, room.operand(X, ldx, tokens, hidden), room.operand(W, ldw, vocab, hidden), targets,
                       target_bytes, loss, lse};
    // tokens of a piece: whole tiles, pieces of one size
    const long long lde = pitch_of(vocab), most = std::max(256ll, kExpBytes / (2 * lde) / 256 * 256);
    const int pieces = static_cast<int>((tokens + most - 1) / most);
    const int piece = static_cast<int>(std::min<long long>(tokens, up((tokens + pieces - 1) / pieces, 256)));
    const int most_chunks = tiles_of(vocab, 64);
    const long long ldh = pitch_of(hidden);
    bf16* e = room.take<bf16>(lde * piece);
    float2* parts = room.take<float2>(static_cast<long long>(most_chunks) * piece);
    float* target_logit = room.take<float>(piece);
    float* factor = room.take<float>(piece);
    bf16* scaled = room.take<bf16>(ldh * piece);
    const long long ld_sum = up(hidden, 4);
    float* sum = piece < tokens ? room.take<float>(ld_sum * vocab) : nullptr;   // of the pieces' dW
    auto products = [&](int t0, int rows, Product (&q)[2]) {
        q[0] = {};
        q[0].a = {e, lde, rows, vocab};
        q[0].b = n.w;
        q[0].b_mn = true;
        q[0].M = rows;
        q[0].N = hidden;
        q[0].out = static_cast<bf16*>(dX) + static_cast<long long>(t0) * ld_dx;
        q[0].ldo = ld_dx;
        q[0].factor = factor;
        const bool last = t0 + rows == tokens;
        q[1] = {};
        q[1].a = {e, lde, rows, vocab, true};
        q[1].b = {scaled, ldh, rows, hidden, true};
        q[1].a_mn = q[1].b_mn = true;
        q[1].M = vocab;
        q[1].N = hidden;
        q[1].f32 = last ? f32 : 1;
        q[1].out = last ? dW : sum;
        q[1].ldo = last ? ld_dw : ld_sum;
        q[1].plus = t0 ? sum : nullptr;
        q[1].ld_plus = ld_sum;
    };
    // room for the products' sums: one piece's product after another's, the last piece may be the shorter one
    const size_t at = room.used;
    size_t end = at;
    for (int i = 0; i < 2; ++i) {
        const int t0 = i ? tokens - 1 - (tokens - 1) % piece : 0;
        Product q[2];
        products(t0, std::min(piece, tokens - t0), q);
        Launches both = arrange(q, 2, g.sms);
        reserve(room, both);
        end = std::max(end, room.used);
        room.used = at;
    }
    room.used = end;
    if ((st = enough(room, workspace_bytes))) return st;
    const auto lock = library_lock();
    if (room.copies.n && (st = status_of(launch_dense_copies(room.copies, stream)))) return st;
    for (long long from = 0; from < tokens; from += piece) {   // (the end of the last piece may pass 32 bits)
        const int t0 = static_cast<int>(from), rows = std::min(piece, tokens - t0);
        int chunk;
        if ((st = entropy_pairs(n, t0, rows, e, lde, parts, target_logit, &chunk, g))) return st;
        EntropyRows r = entropy_rows(n, t0, rows, tiles_of(vocab, chunk), chunk, parts, target_logit);
        r.grad = grad + t0;
        r.e = e;
        r.ld_e = lde;
        r.factor = factor;
        r.scaled = scaled;
        r.ld_scaled = ldh;
        if ((st = status_of(launch_entropy_rows(r, stream)))) return st;
        Product q[2];
        products(t0, rows, q);
        room.used = at;
        Launches both = arrange(q, 2, g.sms);
        reserve(room, both);
        if ((st = run(both, g))) return st;
    }
    return TCL_OK;
}

int tcl_grad_norm(int count, const void* const* tensors, const long long* lengths, const int* types, float* norm,
                  void* workspace, size_t* workspace_bytes, cudaStream_t stream) {
    if (const int st = clip_checks(count, tensors, lengths, types, norm)) return st;
    if (!workspace_bytes || (*workspace_bytes && !workspace)) return TCL_ERR_NULL;
    if (!on(workspace, 256)) return TCL_ERR_ALIGN;
    Gpu g;
    if (const int st = gpu_of(stream, &g)) return st;
    int blocks = 0;
    each_launch(count, tensors, nullptr, lengths, types, [&](const ClipTensors& a) {
        blocks += clip_blocks(a.pieces);
        return TCL_OK;
    });
    Room room{static_cast<uint8_t*>(workspace), *workspace_bytes};
    double* parts = room.take<double>(blocks);
    if (const int st = enough(room, workspace_bytes)) return st;
    int at = 0;
    const int st = each_launch(count, tensors, nullptr, lengths, types, [&](const ClipTensors& a) {
        const int mine = at;
        at += clip_blocks(a.pieces);
        return status_of(launch_square_sums(a, parts + mine, stream));
    });
    return st ? st : status_of(launch_norm(parts, blocks, norm, stream));
}

int tcl_clip_gradients(int count, const void* const* from, void* const* to, const long long* lengths, const int* types,
                       float bound, float* norm, void* workspace, size_t* workspace_bytes, cudaStream_t stream) {
    if (const int st = clip_checks(count, from, lengths, types, norm)) return st;
    if (!(bound >= 0.0f)) return TCL_ERR_CONFIG;
    if (!workspace_bytes || (*workspace_bytes && !workspace) || (count && !to)) return TCL_ERR_NULL;
    if (!on(workspace, 256)) return TCL_ERR_ALIGN;
    for (int i = 0; i < count; ++i) {
        if (lengths[i] && !to[i]) return TCL_ERR_NULL;
        if (!on(to[i], types[i] == TCL_OUT_F32 ? 4 : 2)) return TCL_ERR_ALIGN;
    }
    if (const int st = overlap_checks(count, from, to, lengths, types)) return st;
    Gpu g;
    if (const int st = gpu_of(stream, &g)) return st;
    int blocks = 0;
    each_launch(count, from, to, lengths, types, [&](const ClipTensors& a) {
        blocks += clip_blocks(a.pieces);
        return TCL_OK;
    });
    Room room{static_cast<uint8_t*>(workspace), *workspace_bytes};
    double* parts = room.take<double>(blocks);
    if (const int st = enough(room, workspace_bytes)) return st;
    int at = 0;
    int st = each_launch(count, from, to, lengths, types, [&](const ClipTensors& a) {
        const int mine = at;
        at += clip_blocks(a.pieces);
        return status_of(launch_square_sums(a, parts + mine, stream));
    });
    if (st) return st;
    if (!blocks) return status_of(launch_norm(parts, 0, norm, stream));
    float* told = norm;   // (the first launch's)
    return each_launch(count, from, to, lengths, types, [&](const ClipTensors& a) {
        float* const mine = told;
        told = nullptr;
        return status_of(launch_clip(a, parts, blocks, bound, mine, stream));
    });
}

}  // extern "C"
