// kq_attn_inst.hip -- the attention kernels of one head size, 32 * KQ_ATTN_NB.
#include "kq_attn.h"

namespace kq {
namespace kv {

template <int NB> int launch_attn(bool q8, const Cache &c, const Attn &a, hipStream_t st) {
    const int groups = (a.rows_cap + 16 * a.row_tiles - 1) / (16 * a.row_tiles);
    const int64_t units = (int64_t)a.items * c.kv_heads, grid = (units + 7) / 8 * 8 * groups;
    void (*kern)(Cache, Attn) = q8 ? attn_kernel<true, NB> : attn_kernel<false, NB>;
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(ATTN_THREADS), 0, st, c, a);
    if (a.items > a.B)
        hipLaunchKernelGGL(attn_join_kernel<NB>, dim3((unsigned)(a.B * c.kv_heads * a.rows_cap)), dim3(ATTN_THREADS), 0,
                           st, c, a);
    return launched();
}

template int launch_attn<KQ_ATTN_NB>(bool, const Cache &, const Attn &, hipStream_t);

} // namespace kv
} // namespace kq
