// Instantiates and launches the dense products of few tokens.
#include "dense_launch.cuh"

namespace tcl {
namespace {

template <int BQ, DenseEnd E>
cudaError_t prepare(int* dev) {
    // the shared-memory opt-in is per function and device: set once per device
    static bool attr_done[64] = {};
    cudaError_t err = cudaGetDevice(dev);
    if (err != cudaSuccess) return err;
    if (*dev < 0 || *dev >= 64 || !attr_done[*dev]) {
        err = cudaFuncSetAttribute(dense_few_kernel<BQ, E>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   DenseFewCfg<BQ, E>::SMEM_BYTES);
        if (err == cudaSuccess && *dev >= 0 && *dev < 64) attr_done[*dev] = true;
    }
    return err;
}

template <int BQ, DenseEnd E>
cudaLaunchConfig_t config(int grid, int split, cudaStream_t stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(DenseFewCfg<BQ, E>::THREADS);
    cfg.dynamicSmemBytes = DenseFewCfg<BQ, E>::SMEM_BYTES;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cfg;
}

template <int BQ, DenseEnd E>
cudaError_t launch(const DenseFewLaunch& a) {
    int dev = 0;
    const cudaError_t err = prepare<BQ, E>(&dev);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config<BQ, E>(a.grid, a.p.split, a.stream, attr);
    return cudaLaunchKernelEx(&cfg, dense_few_kernel<BQ, E>, a.w[0], a.w[1], a.x, a.p);
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

int dense_few_clusters(int split, int sms) {
    // (one CTA of any of these kernels fills an SM, so one of them answers for all; asked once per device)
    if (split == 1) return sms;
    static int known[64][4] = {};
    int dev = 0, n = 0;
    if (prepare<16, DenseEnd::STORE>(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sms / split * 3 / 4;
    const int k = split == 2 ? 1 : split == 4 ? 2 : 3;
    if (known[dev][k]) return known[dev][k];
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config<16, DenseEnd::STORE>(split, split, nullptr, attr);
    if (cudaOccupancyMaxActiveClusters(&n, dense_few_kernel<16, DenseEnd::STORE>, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return sms / split * 3 / 4;
    }
    return known[dev][k] = n;
}

cudaError_t launch_dense_few(const DenseFewLaunch& a) {
    switch (a.bq) {
        case 16: return launch<16>(a);
        case 32: return launch<32>(a);
        case 64: return launch<64>(a);
        default: return launch<128>(a);
    }
}

}  // namespace tcl
