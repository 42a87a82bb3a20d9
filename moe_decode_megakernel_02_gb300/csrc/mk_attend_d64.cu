// mk_attend_d64.cu -- the attention kernels for head_dim 64
#include "mk_attend.cuh"

namespace mkop {
int attend_64(const Kind& k, const AttendP* p, KindInfo* info, int grid, bool after, cudaStream_t s) {
    return attend_d<64>(k, p, info, grid, after, s);
}
int join_64(const JoinP& j, cudaStream_t s) { return join_d<64>(j, s); }
}  // namespace mkop
