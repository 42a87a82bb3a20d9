// mk_attend_d256.cu -- the attention kernels for head_dim 256
#include "mk_attend.cuh"

namespace mkop {
int attend_256(const Kind& k, const AttendP* p, KindInfo* info, int grid, bool after, cudaStream_t s) {
    return attend_d<256>(k, p, info, grid, after, s);
}
int join_256(const JoinP& j, cudaStream_t s) { return join_d<256>(j, s); }
}  // namespace mkop
