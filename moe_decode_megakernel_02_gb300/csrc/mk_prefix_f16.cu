// mk_prefix_f16.cu -- the kernels of mk_prefix.cuh for fp16 queries
#include "mk_prefix.cuh"

namespace mkop {

int prefix_f16(int head_dim, int format, const AttendP* p, int grid, cudaStream_t s) {
    return head_dim == 64 ? prefix_pick<64, true>(format, p, grid, s) : prefix_pick<128, true>(format, p, grid, s);
}

}  // namespace mkop
