// Instantiates and launches the scaled e4m3 products.
#include "fp8_launch.cuh"

namespace tcl {
namespace {

template <int BQ, bool PAIR, bool SWAP, bool QVEC>
cudaError_t launch(const Fp8Launch& a) {
    using C = Fp8Cfg<BQ, PAIR, SWAP, QVEC>;
    auto kern = fp8_gemm_kernel<BQ, PAIR, SWAP, QVEC>;
    // the shared-memory opt-in is per function and device: set once per device
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
        if (err != cudaSuccess) return err;
        if (dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    const int cluster = PAIR ? C::CTAS : a.p.split;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a.tmP, a.tmQ, a.tmC, a.p);
}

template <int BQ, bool PAIR, bool SWAP, bool QVEC>
Fp8TileInfo info() {
    using C = Fp8Cfg<BQ, PAIR, SWAP, QVEC>;
    return {C::BP, C::BQ, C::CTAS, 128, C::BQL, SWAP ? 1 : 0, C::PER_SM};
}

}  // namespace

Fp8TileInfo fp8_tile_info(Fp8Tile t) {
    switch (t) {
        case Fp8Tile::FEW16: return info<16, false, true, true>();
        case Fp8Tile::FEW32: return info<32, false, true, true>();
        case Fp8Tile::PAIR: return info<256, true, false, true>();
        default: return info<128, false, false, true>();
    }
}

cudaError_t launch_fp8_gemm(const Fp8Launch& a) {
    const bool blocks = a.p.Q.block != 0;   // (few tokens: Q is the tokens' side, whose scales belong to rows)
    switch (a.tile) {
        case Fp8Tile::FEW16: return launch<16, false, true, true>(a);
        case Fp8Tile::FEW32: return launch<32, false, true, true>(a);
        case Fp8Tile::PAIR: return blocks ? launch<256, true, false, false>(a) : launch<256, true, false, true>(a);
        default: return blocks ? launch<128, false, false, false>(a) : launch<128, false, false, true>(a);
    }
}

}  // namespace tcl
