// grouped.cu -- the compiled variants of the grouped products.
#include "grouped_kernel.cuh"

#include <atomic>

#include "experts.h"

namespace gp {
namespace {

template <class Cfg>
cudaError_t prepare(int *dev_out)
{
    static std::atomic<int> done[128];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    if (!done[dev].load()) {
        e = cudaFuncSetAttribute(grouped_kernel<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        done[dev].store(1);
    }
    *dev_out = dev;
    return cudaSuccess;
}

template <class Cfg>
void configure(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int grid, cudaStream_t s)
{
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = Cfg::CLUSTER;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = Cfg::PAIR ? 2 : 1;
}

template <class Cfg>
cudaError_t launch(const GroupedMaps &maps, const GroupedParams &p, int grid, cudaStream_t s)
{
    int dev = 0;
    cudaError_t e = prepare<Cfg>(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    configure<Cfg>(cfg, attr, grid, s);
    e = cudaLaunchKernelEx(&cfg, grouped_kernel<Cfg>, maps, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <class Cfg>
int max_units()
{
    static std::atomic<int> cache[128];
    int dev = 0;
    if (prepare<Cfg>(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    int n = cache[dev].load();
    if (n > 0) return n;
    int sms = 0;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if constexpr (Cfg::PAIR) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        configure<Cfg>(cfg, attr, Cfg::CLUSTER * (sms / Cfg::CLUSTER), nullptr);
        cfg.attrs = attr + 1;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, grouped_kernel<Cfg>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
    } else {
        n = sms;
    }
    cache[dev].store(n);
    return n;
}

template <class Cfg>
constexpr GroupedVariant variant()
{
    return GroupedVariant{Cfg::MODE, Cfg::BN, Cfg::TILE_F, Cfg::PAIR ? 1 : 0, Cfg::CTA_BN, Cfg::BK, Cfg::B_PART_ROWS, Cfg::SMEM_BYTES, &launch<Cfg>,
                          &max_units<Cfg>};
}

const GroupedVariant kVariants[] = {
    variant<GroupedCfg<kRows, 32, false, 128, 64>>(),
    variant<GroupedCfg<kRows, 32, false, 128>>(),  variant<GroupedCfg<kRows, 64, false, 128>>(),
    variant<GroupedCfg<kRows, 128, false>>(), variant<GroupedCfg<kRows, 256, true>>(),
    variant<GroupedCfg<kRowsT, 32, false, 128>>(), variant<GroupedCfg<kRowsT, 64, false, 128>>(),
    variant<GroupedCfg<kRowsT, 128, false>>(), variant<GroupedCfg<kRowsT, 256, true>>(),
    variant<GroupedCfg<kWeights, 256, true>>(),
};

}  // namespace

const GroupedVariant *grouped_variant(int mode, int bn, int tile_f)
{
    for (const GroupedVariant &v : kVariants)
        if (v.mode == mode && v.bn == bn && v.tile_f == tile_f) return &v;
    return nullptr;
}

}  // namespace gp
