// mk_prefix.cu -- the kernels of mk_prefix.cuh for bf16 queries
#include "mk_prefix.cuh"

namespace mkop {

int prefix_bf16(int head_dim, int format, const AttendP* p, int grid, cudaStream_t s) {
    return head_dim == 64 ? prefix_pick<64, false>(format, p, grid, s) : prefix_pick<128, false>(format, p, grid, s);
}

}  // namespace mkop
