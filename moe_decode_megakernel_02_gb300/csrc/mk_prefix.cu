// mk_prefix.cu -- launches of the shared-prefix kernels (mk_prefix.cuh)
#include "mk_prefix.cuh"

namespace mkop {

namespace {

// K or V as a 4-D tensor; a box is up to 64 rows of a page by 64 values, in
// the 128-byte swizzled order the products read
int map_of(const AttendP& p, const void* base, int head_dim, CUtensorMap* out) {
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (Encode) nullptr;
        return (Encode)f;
    }();
    if (!encode) return fail(MK_ERR_CUDA, "attend: the driver has no cuTensorMapEncodeTiled");
    const cuuint32_t rows = 1u << p.ps_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)head_dim, rows, (cuuint64_t)p.H, (cuuint64_t)p.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.row_b, (cuuint64_t)p.head_b, (cuuint64_t)p.page_b};
    const cuuint32_t box[4] = {64, rows < 64 ? rows : 64, 1, 1}, one[4] = {1, 1, 1, 1};
    const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, one,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(MK_ERR_CUDA, "attend: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return MK_OK;
}

template <int D, int FMT>
int run(const AttendP* p, int grid, cudaStream_t s) {
    using S = PrefixShape<D, FMT>;
    auto kern = prefix_kernel<D, FMT>;
    if (!p) return cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM), "mk_pages_attend");
    PrefixMaps maps = {};
    if constexpr (FMT == MK_KV_BF16) {
        if (const int rc = map_of(*p, p->k, D, &maps.k)) return rc;
        if (const int rc = map_of(*p, p->v, D, &maps.v)) return rc;
    }
    kern<<<grid, S::NT, S::SMEM, s>>>(*p, maps);
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
