// mk_prefix.cu -- launches of the shared-prefix kernels (mk_prefix.cuh)
#include "mk_prefix.cuh"

namespace mkop {

namespace {
template <int D, int FMT>
int run(const AttendP* p, int grid, cudaStream_t s) {
    using S = PrefixShape<D, FMT>;
    auto kern = prefix_kernel<D, FMT>;
    if (!p) return cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM), "mk_pages_attend");
    kern<<<grid, S::NT, S::SMEM, s>>>(*p);
    return cuda_status(cudaGetLastError(), "mk_pages_attend");
}
template <int D>
int run_d(int format, const AttendP* p, int grid, cudaStream_t s) {
    if (format == MK_KV_E4M3) return run<D, MK_KV_E4M3>(p, grid, s);
    if (format == MK_KV_INT8) return run<D, MK_KV_INT8>(p, grid, s);
    return run<D, MK_KV_BF16>(p, grid, s);
}
}  // namespace

int prefix_run(int head_dim, int format, const AttendP* p, int grid, cudaStream_t s) {
    return head_dim == 64 ? run_d<64>(format, p, grid, s) : run_d<128>(format, p, grid, s);
}

}  // namespace mkop
