// attend_paged.cu -- hca_attend_paged: dense attention over the visible entries
// of a paged cache plus a ring of window rows per sequence.
//
// Two kernels share the key set: the entries that all requests share
// (attend_prefix.cu, one product for the whole batch) and every request's own
// entries and window (the gather kernel of attend_tc.cu).  Each leaves partial
// rows O = sum_j 2^(s_j - m) x_j with their (m, l); the merge here weighs them
// in a fixed order (the sum and the row are held in 32 bits: the one rounding
// is that of the output):
//   out = sum_i 2^(m_i - M) O_i / (sum_i 2^(m_i - M) l_i + sink)
#include <algorithm>

#include "attend_common.cuh"
#include "common.cuh"
#include "kernels.h"

namespace csa {

void attend_tc_plan(long long n_bq, int H, long long max_keys, int *splits, long long *kps);
int launch_attend_tc(AttendArgs a, const DevCtx &ctx, cudaStream_t st, bool pdl);

namespace {

constexpr int kMergeThreads = 256;

struct MergeArgs {
    AttendArgs a;
    PrefixPlan plan;  // pairs == 0: no shared entries
    const float *part;
    const float2 *ml;
};

// A warp: 4 rows x 64 dims, a thread 8 dims of one row (32 bytes of each partial;
// a partial's 4 rows x 8 dims are 128 contiguous bytes in the prefix layout).
__global__ void __launch_bounds__(kMergeThreads) attend_merge_kernel(const MergeArgs g) {
    const AttendArgs &a = g.a;
    const int slabs = a.D / 64, lane = threadIdx.x & 31;
    const long long wid = (long long)blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
    const int slab = (int)(wid % slabs);
    const long long row = wid / slabs * 4 + (lane >> 3), n_rows = a.n_bq * a.H;  // row = bq * H + h
    const bool active = row < n_rows;  // no early exit: the rotation's shuffles need whole warps
    const int d0 = slab * 64 + (lane & 7) * 8;
    const long long bq = active ? row / a.H : 0;
    const int h = active ? (int)(row - bq * a.H) : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int p0 = 0, np = 0;
    const float4 *psrc = nullptr;
    const float2 *pml = nullptr;
    const int DP = prefix_dims(a.D);
    if (g.plan.pairs > 0 && active) {
        const int rt = (int)(row / kPrefixRows), rr = (int)(row % kPrefixRows);
        p0 = g.plan.pair_of((long long)rt * g.plan.key_tiles);
        np = g.plan.pair_of((long long)(rt + 1) * g.plan.key_tiles - 1) - p0 + 1;
        pml = g.ml + (size_t)(p0 + rt) * kPrefixRows + rr;
        // dim d0 of row rr: [rank][piece of 8 columns][lane half x 64 rows][8]
        const int hf = d0 / (DP / 2), col = d0 % (DP / 2);
        psrc = reinterpret_cast<const float4 *>(g.part) +
               (((size_t)(p0 + rt) * 2 + (rr >> 6)) * (DP / 16) * 128 + (size_t)(col / 8) * 128 + hf * 64 + (rr & 63)) * 2;
    }
    const size_t pstride = (size_t)kPrefixRows * DP / 4;  // float4 per prefix partial
    const size_t own_rows = (size_t)n_rows;
    const float2 *oml = a.part_ml + (active ? row : 0);
    const float4 *osrc = reinterpret_cast<const float4 *>(a.part_f + (size_t)bq * a.H * a.D);
    int ostep = 1;
    if (a.part_perm) {
        osrc += ((size_t)(h >> 6) * slabs + slab) * 1024 + ((h & 63) >> 4) * 256 + ((d0 & 31) / 4) * 32 + (h & 15) +
                ((d0 >> 5) & 1) * 16;
        ostep = 32;
    } else {
        osrc += ((size_t)h * a.D + d0) / 4;
    }
    const size_t ostride = own_rows * a.D / 4;
    float M = -INFINITY;
    for (int i = 0; i < np; ++i) M = fmaxf(M, pml[(size_t)i * kPrefixRows].x);
    if (active)
        for (int i = 0; i < a.splits; ++i) M = fmaxf(M, oml[i * own_rows].x);
    float L = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const auto add = [&](const float2 ml, const float4 *src, int step) {
        if (ml.x == -INFINITY) return;  // no key: nothing was written
        const float w = exp2f(ml.x - M);
        const float4 x = src[0], y = src[step];
        L = fmaf(w, ml.y, L);
        acc[0] = fmaf(w, x.x, acc[0]); acc[1] = fmaf(w, x.y, acc[1]);
        acc[2] = fmaf(w, x.z, acc[2]); acc[3] = fmaf(w, x.w, acc[3]);
        acc[4] = fmaf(w, y.x, acc[4]); acc[5] = fmaf(w, y.y, acc[5]);
        acc[6] = fmaf(w, y.z, acc[6]); acc[7] = fmaf(w, y.w, acc[7]);
    };
#pragma unroll 4
    for (int i = 0; i < np; ++i) add(pml[(size_t)i * kPrefixRows], psrc + i * pstride, 1);
    if (active) {
#pragma unroll 4
        for (int i = 0; i < a.splits; ++i) add(oml[i * own_rows], osrc + i * ostride, ostep);
    }
    if (a.sinks && active) L += exp2f(__ldg(a.sinks + h) * 1.4426950408889634f - M);
    const float inv = L > 0.f ? 1.0f / L : 0.f;
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = acc[e] * inv;
    if (a.rope_cos) {
        // conjugate rotation of the trailing 64 channels: channel D-64+j pairs with
        // D-32+j, held by the thread 4 lanes away
        float pv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) pv[e] = __shfl_xor_sync(0xffffffffu, o[e], 4);
        if (slab == slabs - 1 && active) {
            const long long t = __ldg(a.q_pos + bq);
            const bool first = (lane & 4) == 0;
            const int i0 = (lane & 3) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 cs = rope_cs(a, t, i0 + e);
                o[e] = first ? o[e] * cs.x + pv[e] * cs.y : o[e] * cs.x - pv[e] * cs.y;
            }
        }
    }
    if (active) *reinterpret_cast<uint4 *>(a.out + (size_t)row * a.D + d0) = pack8(o);
}

// How a call splits its keys, and where its partial rows lie in the workspace.
struct PagedPlan {
    PrefixPlan prefix;  // pairs == 0: every key by the gather kernel
    int splits;
    long long keys_per_split;
    size_t keys, part, ml, own, own_ml, bytes;  // offsets
};

size_t take(size_t &at, size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~size_t(255);
    return o;
}

PagedPlan paged_plan(long long n_bq, int H, int D, int page, int max_pages, long long n_shared, int W, bool fp8) {
    PagedPlan pl = {};
    const long long rows = n_bq * H, cap = (long long)max_pages * page;
    const bool prefix = n_shared > 0 && rows <= 0x7fffffffLL;
    size_t at = 0;
    if (prefix) {
        pl.prefix = prefix_plan(rows, n_shared);
        if (fp8) pl.keys = take(at, (size_t)n_shared * D * sizeof(uint16_t));
        pl.part = take(at, (size_t)pl.prefix.partials() * kPrefixRows * prefix_dims(D) * sizeof(float));
        pl.ml = take(at, (size_t)pl.prefix.partials() * kPrefixRows * sizeof(float2));
    }
    attend_tc_plan(n_bq, H, (prefix ? cap - n_shared : cap) + W, &pl.splits, &pl.keys_per_split);
    if (prefix || pl.splits > 1) {
        pl.own = take(at, (size_t)pl.splits * rows * D * sizeof(float));
        pl.own_ml = take(at, (size_t)pl.splits * rows * sizeof(float2));
    }
    pl.bytes = at;
    return pl;
}

}  // namespace

size_t attend_paged_workspace_bytes(int batch, int nq, int H, int D, int page, int max_pages, long long n_shared, int W,
                                    bool fp8) {
    return paged_plan((long long)batch * nq, H, D, page, max_pages, n_shared, W, fp8).bytes;
}

int launch_attend_paged(const PagedArgs &p, void *ws, size_t ws_bytes, const DevCtx &ctx, cudaStream_t st) {
    const bool fp8 = p.fp8.kv != nullptr;
    AttendArgs a = {};
    a.q = p.q; a.q_gain = p.q_gain; a.sinks = p.sinks; a.rope_cos = p.rope_cos; a.rope_sin = p.rope_sin;
    a.rope_npos = p.rope_npos;
    a.kv = p.pool; a.kv8 = p.fp8.kv; a.kv8e = p.fp8.kv_exp;
    a.win = p.ring; a.win8 = p.fp8.win; a.win8e = p.fp8.win_exp;
    a.N = (long long)p.max_pages * p.page; a.m = p.m; a.dense = true;
    a.table = p.table; a.max_pages = p.max_pages; a.page = p.page; a.n_pages = p.n_pages;
    a.win_rows = p.ring_rows; a.W = p.W; a.q_pos = p.q_pos; a.nq = p.nq; a.n_bq = (long long)p.batch * p.nq;
    a.H = p.H; a.D = p.D; a.scale = p.scale; a.eps = p.eps; a.out = p.out;
    const PagedPlan pl = paged_plan(a.n_bq, a.H, a.D, a.page, a.max_pages, p.n_shared, a.W, fp8);
    if (pl.bytes > 0 && (!ws || ws_bytes < pl.bytes)) return CSA_ERR_WORKSPACE;
    char *w = static_cast<char *>(ws);
    const bool prefix = pl.prefix.pairs > 0;
    a.splits = pl.splits;
    a.keys_per_split = pl.keys_per_split;
    MergeArgs g = {};
    if (prefix) {
        PrefixArgs x = {};
        x.a = a;
        x.plan = pl.prefix;
        x.n_shared = p.n_shared;
        x.keys = p.pool;
        x.linear = fp8;
        if (fp8) {
            uint16_t *keys = reinterpret_cast<uint16_t *>(w + pl.keys);
            const int rc = launch_prefix_rows(a.kv8, a.kv8e, a.table, a.page, a.n_pages, a.D, p.n_shared, keys, st);
            if (rc != CSA_OK) return rc;
            x.keys = keys;
        }
        x.part = reinterpret_cast<float *>(w + pl.part);
        x.ml = reinterpret_cast<float2 *>(w + pl.ml);
        const int rc = launch_attend_prefix(x, ctx, st);
        if (rc != CSA_OK) return rc;
        a.e_first = p.n_shared;
        g.plan = pl.prefix;
        g.part = x.part;
        g.ml = x.ml;
    }
    const bool merge = prefix || pl.splits > 1;
    if (merge) {
        a.part_f = reinterpret_cast<float *>(w + pl.own);
        a.part_ml = reinterpret_cast<float2 *>(w + pl.own_ml);
        a.part_perm = a.H % 64 == 0 ? 1 : 0;
    }
    const int rc = launch_attend_tc(a, ctx, st, prefix);
    if (rc != CSA_OK || !merge) return rc;
    g.a = a;
    const long long warps = (a.n_bq * a.H + 3) / 4 * (a.D / 64);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((warps + kMergeThreads / 32 - 1) / (kMergeThreads / 32)));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_merge_kernel, g) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // namespace csa
