// few_bf16.cu -- the kernels for a few rows, bf16.
#include "few_kernel.cuh"

namespace gp {

cudaError_t launch_few_bf16(const FewLaunch &l, const FewParams &p, cudaStream_t s)
{
    return l.four ? launch_few_type<true, true>(l, p, s) : launch_few_type<true, false>(l, p, s);
}

int few_room(int one, int split)
{
    static std::atomic<int> rooms[128][2][9];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128 || split < 1 || split > 8) return 0;
    std::atomic<int> &room = rooms[dev][one ? 1 : 0][split];
    if (room.load() == 0) room.store(one ? few_room_of<4>(split) : few_room_of<1>(split));
    return room.load();
}

}  // namespace gp
