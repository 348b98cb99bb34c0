// attend_paged.cu -- hca_attend_paged: dense attention over the visible entries
// of a paged cache plus a ring of window rows per sequence.
#include <algorithm>

#include "attend_common.cuh"
#include "common.cuh"
#include "kernels.h"

namespace csa {

void attend_tc_plan(long long n_bq, int H, long long max_keys, int *splits, long long *kps);
int launch_attend_tc(AttendArgs a, const DevCtx &ctx, cudaStream_t st, bool pdl);

size_t attend_paged_workspace_bytes(int batch, int nq, int H, int D, int page, int max_pages, long long n_shared, int W,
                                    bool fp8) {
    (void)n_shared;
    (void)fp8;
    return attend_workspace_bytes(batch, nq, H, D, (long long)max_pages * page + W);
}

int launch_attend_paged(const PagedArgs &p, void *ws, size_t ws_bytes, const DevCtx &ctx, cudaStream_t st) {
    AttendArgs a = {};
    a.q = p.q; a.q_gain = p.q_gain; a.sinks = p.sinks; a.rope_cos = p.rope_cos; a.rope_sin = p.rope_sin;
    a.rope_npos = p.rope_npos;
    a.kv = p.pool; a.kv8 = p.fp8.kv; a.kv8e = p.fp8.kv_exp;
    a.win = p.ring; a.win8 = p.fp8.win; a.win8e = p.fp8.win_exp;
    a.N = (long long)p.max_pages * p.page; a.m = p.m; a.dense = true;
    a.table = p.table; a.max_pages = p.max_pages; a.page = p.page; a.n_pages = p.n_pages; a.e_first = 0;
    a.win_rows = p.ring_rows; a.W = p.W; a.q_pos = p.q_pos; a.nq = p.nq; a.n_bq = (long long)p.batch * p.nq;
    a.H = p.H; a.D = p.D; a.scale = p.scale; a.eps = p.eps; a.out = p.out;
    attend_tc_plan(a.n_bq, a.H, a.N + a.W, &a.splits, &a.keys_per_split);
    if (a.splits > 1) {
        const size_t rows = (size_t)a.splits * a.n_bq * a.H;
        if (!ws || ws_bytes < rows * ((size_t)a.D * sizeof(uint16_t) + sizeof(float2))) return CSA_ERR_WORKSPACE;
        a.part_o = static_cast<uint16_t *>(ws);
        a.part_perm = a.H % 64 == 0 ? 1 : 0;
        a.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(ws) + rows * a.D * sizeof(uint16_t));
    }
    return launch_attend_tc(a, ctx, st, false);
}

}  // namespace csa
