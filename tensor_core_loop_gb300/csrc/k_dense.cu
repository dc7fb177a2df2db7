// Instantiates and launches the dense products on pairs of SMs.
#include "dense_launch.cuh"

namespace tcl {
namespace {

template <int BN, DenseEnd E>
cudaError_t launch(const DenseLaunch& a) {
    using C = DenseCfg<BN>;
    auto kern = dense_pair_kernel<BN, E>;
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
    cfg.gridDim = dim3(2 * a.pairs);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a.maps, a.p);
}

template <int BN>
cudaError_t launch(const DenseLaunch& a) {
    switch (a.end) {
        case DenseEnd::GATE: return launch<BN, DenseEnd::GATE>(a);
        case DenseEnd::GATE_GRAD: return launch<BN, DenseEnd::GATE_GRAD>(a);
        case DenseEnd::ENTROPY: return launch<BN, DenseEnd::ENTROPY>(a);
        default: return launch<BN, DenseEnd::STORE>(a);
    }
}

}  // namespace

cudaError_t launch_dense_pair(const DenseLaunch& a) { return a.bn == 256 ? launch<256>(a) : launch<128>(a); }

}  // namespace tcl
