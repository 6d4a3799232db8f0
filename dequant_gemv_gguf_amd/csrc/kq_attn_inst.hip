// kq_attn_inst.hip -- the attention kernels of one head size, 32 * KQ_ATTN_NB.
#include "kq_attn.h"

namespace kq {
namespace kv {

template <int NB> int launch_attn(bool q8, bool nt, int rt, const Cache &c, const Attn &a, hipStream_t st) {
    const int wg_rows = 16 * rt * a.row_waves, groups = (a.rows_cap + wg_rows - 1) / wg_rows;
    void (*kern)(Cache, Attn) = q8 ? (nt ? attn_kernel<true, NB, true, 1> : attn_kernel<true, NB, false, 1>)
                                   : (nt ? attn_kernel<false, NB, true, 1> : attn_kernel<false, NB, false, 1>);
    if constexpr (NB <= TWO_TILES_NB) {
        if (rt == 2) kern = q8 ? attn_kernel<true, NB, false, 2> : attn_kernel<false, NB, false, 2>;
    }
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

template int launch_attn<KQ_ATTN_NB>(bool, bool, int, const Cache &, const Attn &, hipStream_t);

} // namespace kv
} // namespace kq
