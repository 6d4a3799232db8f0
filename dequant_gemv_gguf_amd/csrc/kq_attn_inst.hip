// kq_attn_inst.hip -- the attention kernels of one head size, 32 * KQ_ATTN_NB.
#include "kq_attn.h"

namespace kq {
namespace kv {

template <int NB> int launch_attn(bool q8, bool nt, const Cache &c, const Attn &a, hipStream_t st) {
    const int groups = (a.rows_cap + 16 * a.row_tiles - 1) / (16 * a.row_tiles);
    void (*kern)(Cache, Attn) = q8 ? (nt ? attn_kernel<true, NB, true> : attn_kernel<true, NB, false>)
                                   : (nt ? attn_kernel<false, NB, true> : attn_kernel<false, NB, false>);
    const unsigned pieces = groups == 1 ? (unsigned)a.items : (unsigned)((a.items + 7) / 8 * 8 * groups);
    hipLaunchKernelGGL(kern, dim3(pieces, (unsigned)c.kv_heads), dim3(ATTN_THREADS), 0, st, c, a);
    if (a.items > a.B) {
        const dim3 grid((unsigned)a.rows_cap, (unsigned)c.kv_heads, (unsigned)a.B);
        // many pieces a row: more threads, so that a thread's pieces are all on their way at once
        if (a.items > 32 * a.B)
            hipLaunchKernelGGL((attn_join_kernel<NB, 1024>), grid, dim3(1024), 0, st, c, a);
        else
            hipLaunchKernelGGL((attn_join_kernel<NB, 256>), grid, dim3(256), 0, st, c, a);
    }
    return launched();
}

template int launch_attn<KQ_ATTN_NB>(bool, bool, const Cache &, const Attn &, hipStream_t);

} // namespace kv
} // namespace kq
