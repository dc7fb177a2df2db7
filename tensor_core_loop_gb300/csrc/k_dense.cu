// Instantiates and launches the dense products on pairs of SMs.
#include "dense_launch.cuh"

namespace tcl {
namespace {

template <bool A_MN, bool B_MN, DenseEnd E>
cudaError_t launch(const DenseLaunch& a) {
    auto kern = dense_pair_kernel<A_MN, B_MN, E>;
    // the shared-memory opt-in is per function and device: set once per device
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, DenseCfg::SMEM_BYTES);
        if (err != cudaSuccess) return err;
        if (dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(DenseCfg::THREADS);
    cfg.dynamicSmemBytes = DenseCfg::SMEM_BYTES;
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
    return cudaLaunchKernelEx(&cfg, kern, a.a[0], a.a[1], a.b[0], a.b[1], a.c[0], a.c[1], a.c[2], a.p);
}

}  // namespace

cudaError_t launch_dense_pair(const DenseLaunch& a) {
    switch (a.end) {
        case DenseEnd::GATE: return launch<false, false, DenseEnd::GATE>(a);
        case DenseEnd::GATE_GRAD: return launch<false, true, DenseEnd::GATE_GRAD>(a);
        case DenseEnd::ENTROPY: return launch<false, false, DenseEnd::ENTROPY>(a);
        default:
            if (a.a_mn) return launch<true, true, DenseEnd::STORE>(a);
            return a.b_mn ? launch<false, true, DenseEnd::STORE>(a) : launch<false, false, DenseEnd::STORE>(a);
    }
}

}  // namespace tcl
