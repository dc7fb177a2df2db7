// Instantiates and launches the dense products of few tokens.
#include "dense_launch.cuh"

namespace tcl {
namespace {

template <int BQ, DenseEnd E>
cudaError_t launch(const DenseFewLaunch& a) {
    using C = DenseFewCfg<BQ, E>;
    auto kern = dense_few_kernel<BQ, E>;
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
    attr[1].val.clusterDim.x = a.p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a.w[0], a.w[1], a.x, a.p);
}

template <int BQ>
cudaError_t launch(const DenseFewLaunch& a) {
    switch (a.end) {
        case DenseEnd::GATE: return launch<BQ, DenseEnd::GATE>(a);
        case DenseEnd::ENTROPY: return launch<BQ, DenseEnd::ENTROPY>(a);
        default: return launch<BQ, DenseEnd::STORE>(a);
    }
}

}  // namespace

int dense_few_per_sm(int bq) { return bq <= 32 ? 2 : 1; }

cudaError_t launch_dense_few(const DenseFewLaunch& a) {
    return a.bq == 16 ? launch<16>(a) : a.bq == 32 ? launch<32>(a) : launch<64>(a);
}

}  // namespace tcl
