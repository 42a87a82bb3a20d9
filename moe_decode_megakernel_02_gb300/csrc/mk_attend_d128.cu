// mk_attend_d128.cu -- the attention kernels for head_dim 128
#include "mk_attend.cuh"

namespace mkop {
int attend_128(const Kind& k, const AttendP* p, KindInfo* info, int grid, bool after, cudaStream_t s) {
    return attend_d<128>(k, p, info, grid, after, s);
}
int join_128(const JoinP& j, cudaStream_t s) { return join_d<128>(j, s); }
}  // namespace mkop
