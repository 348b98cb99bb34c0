// attend_paged.cu -- hca_attend_paged: dense attention over the visible entries
// of a paged cache plus a ring of window rows per sequence.
//
// A batch that shares a prefix takes attend_prefix.cu (all rows stacked), others
// the gather kernel of attend_tc.cu (query by query).  Either leaves partial
// rows O = sum_j 2^(s_j - m) x_j with their (m, l) where the keys of a row are
// split; the merge here weighs them in a fixed order (the sum and the row are
// held in 32 bits: the one rounding is that of the output):
//   out = sum_i 2^(m_i - M) O_i / (sum_i 2^(m_i - M) l_i + sink)
#include <algorithm>

#include "attend_common.cuh"
#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace csa {

int attend_tc_plan(long long n_bq, int H, long long max_keys);
int launch_attend_tc(AttendArgs a, const DevCtx &ctx, cudaStream_t st, bool pdl);

namespace {

constexpr int kMergeThreads = 256;

struct MergeArgs {
    AttendArgs a;
    PrefixPlan plan;  // pairs > 0: the partials of attend_prefix.cu, else the splits of attend_tc.cu
    const float *part;
    const float2 *ml;
    const int2 *meet;
    FastDiv H;
    int n_rows;
    // what attend_prefix.cu worked on (see PrefixArgs): its keys, and the query rows hi + lo with their factors, if
    // they were rewritten (lo null: a.q)
    const uint16_t *keys;
    long long n_shared;
    int own_cap;
    const uint16_t *hi, *lo;
    const float *rq;
};

// Rows of attend_prefix.cu again, without a row tile: its P V takes the keys of all queries of a tile for all of
// their rows, under weights of 0 where a row does not take a key, and 0 x NaN or infinity reaches the row all the
// same.  Such rows (`bad`: NaN in these 8 dims under a sum that is none) are computed anew here, from their own
// keys only, by the whole block: lane i of every warp has row `row` (t < 0: none) with 8 dims from d0 on, the
// warps take the scores of four keys each at a time, the threads with `bad` their dims.  A row whose own keys make
// it NaN (an infinity under a score of -inf) gets it again.  In 32 bits, at its leisure: 96 requests of 16 heads over
// 16K entries take 5.8 ms instead of 43 us if one request's window holds an infinity, but nothing else gets here.
// (Looking through the keys before P V instead, 16 KiB a tile and SM, took 9 us of every such call.)
constexpr int kRedoEach = 4, kRedoKeys = kRedoEach * (kMergeThreads / 32);  // keys of a warp, of the block
constexpr uint32_t kNoKey = 0xffffffffu, kRingKey = 0x80000000u;

// whether queries share the row tile of this row
CSA_DEVINL bool shares_row_tile(const MergeArgs &g, int row) {
    const int first = row / kPrefixRows * kPrefixRows;
    return g.H.div(first) != g.H.div(std::min(first + kPrefixRows, g.n_rows) - 1);
}

__device__ __noinline__ void redo_rows(const MergeArgs &g, int row, bool active, bool bad, int d0, float *out) {
    const AttendArgs &a = g.a;
    __shared__ float score[kRedoKeys][32];
    __shared__ uint32_t place[kRedoKeys][32];  // row of the pool, the copy or (kRingKey) the rings
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int bq = active ? g.H.div(row) : 0, h = row - bq * a.H;
    const long long t = active ? __ldg(a.q_pos + bq) : -1, b = bq / a.nq;
    const long long entries = n_visible(t, a.m, a.N), u0 = t - a.W + 1 > 0 ? t - a.W + 1 : 0;
    const long long n = t < 0 ? 0 : entries + (t - u0 + 1);
    const uint16_t *hi = (g.lo ? g.hi : a.q) + (size_t)(active ? row : 0) * a.D;
    const uint16_t *lo = g.lo ? g.lo + (size_t)(active ? row : 0) * a.D : nullptr;
    float factor;
    if (g.lo) {
        factor = active ? __ldg(g.rq + row) : 0.f;
    } else {
        float ss = 0.f;
#pragma unroll 1
        for (int d = 0; d < a.D; d += 8) {
            float q[8];
            unpack8(ldg16(hi + d), q);
            for (int e = 0; e < 8; ++e) ss = fmaf(q[e], q[e], ss);
        }
        factor = (1.0f / sqrtf(ss / (float)a.D + a.eps)) * a.scale * 1.4426950408889634f;
    }
    const uint16_t *rings = g.own_cap >= 0 ? g.keys + (g.n_shared + a.n_bq / a.nq * g.own_cap) * a.D : a.win;
    const auto values = [&](uint32_t at) { return at & kRingKey ? rings + (size_t)(at & ~kRingKey) * a.D : g.keys + (size_t)at * a.D; };
    float M = -INFINITY, L = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    // (every warp has the same rows, so that the loop ends for all of them together)
    for (long long k0 = 0; __any_sync(0xffffffffu, k0 < n); k0 += kRedoKeys) {
        __syncthreads();
        const uint16_t *x[kRedoEach];
#pragma unroll
        for (int i = 0; i < kRedoEach; ++i) {
            const long long k = k0 + kRedoEach * warp + i;
            uint32_t at = kNoKey;
            if (k < n && k >= entries) {
                at = kRingKey | (uint32_t)(b * a.win_rows + (u0 + (k - entries)) % a.win_rows);
            } else if (k < n) {
                const bool shared = k < g.n_shared;
                const int id = __ldg(a.table + (shared ? 0 : b * a.max_pages) + k / a.page);
                if (id < 0 || id >= a.n_pages) {  // (the copy has zeros there)
                } else if (g.own_cap >= 0) {
                    at = (uint32_t)(shared ? k : g.n_shared + b * g.own_cap + (k - g.n_shared));
                } else {
                    at = (uint32_t)((long long)id * a.page + k % a.page);
                }
            }
            place[kRedoEach * warp + i][lane] = at;
            x[i] = at == kNoKey ? hi : values(at);  // (a score that is not used)
        }
        float s[kRedoEach] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int d = 0; d < a.D; d += 8) {
            float q[8];
            unpack8(ldg16(hi + d), q);
            if (lo) {
                float l[8];
                unpack8(ldg16(lo + d), l);
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] += l[e];
            }
#pragma unroll
            for (int i = 0; i < kRedoEach; ++i) {
                float y[8];
                unpack8(ldg16(x[i] + d), y);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[i] = fmaf(q[e], y[e], s[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kRedoEach; ++i) score[kRedoEach * warp + i][lane] = s[i] * factor;
        __syncthreads();
        if (bad)
#pragma unroll 4
            for (int i = 0; i < kRedoKeys; ++i) {
                const uint32_t at = place[i][lane];
                if (at == kNoKey) continue;
                const float s = score[i][lane];
                if (s > M) {
                    const float f = exp2f(M - s);
                    L *= f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] *= f;
                    M = s;
                }
                const float p = s == -INFINITY ? 0.f : exp2f(s - M);
                L += p;
                float x[8];
                unpack8(ldg16(values(at) + d0), x);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = fmaf(p, x[e], acc[e]);
            }
    }
    if (!bad) return;
    M = fmaxf(M, kLowest);  // (it has keys)
    if (a.sinks) L += exp2f(__ldg(a.sinks + h) * 1.4426950408889634f - M);
    const float inv = inverse_sum(M, L);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = acc[e] * inv;
}

// A block: 32 rows x 64 dims; a warp 8 of the dims, a lane one row: two 16-byte pieces of each
// partial, 512 contiguous bytes a load, kAtOnce partials in flight; the output goes through
// shared memory (its rows are contiguous the other way).  Bound by the partials' bytes: 27 MB of
// 32 x 128 rows of 512 dims in ~5 us (lanes along the dims, 64-byte pieces of the partials: 8.4 us).
// Rows of two or three partials want warps, those of a dozen want loads in flight.
// kGroups = 4, for few rows of many partials: a block 32 rows x 2 x 8 dims (those that RoPE
// pairs), four warps a quarter of the partials each; their sums meet in shared memory.
// kRedo: rows of several queries share the row tiles of attend_prefix.cu (redo_rows).
template <int kAtOnce, int kGroups, bool kRedo>
__global__ void __launch_bounds__(kMergeThreads, kAtOnce <= 2 ? 4 : 2) attend_merge_kernel(const __grid_constant__ MergeArgs g) {
    const AttendArgs &a = g.a;
    __shared__ float tile[32][65];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slab_bits = 31 - __clz(a.D / 64);  // D is 64 .. 512, a power of two
    constexpr int kSlices = 8 / kGroups;  // of 8 dims, in a block
    const int slice = warp % kSlices, group = warp / kSlices;
    const int sub = (int)blockIdx.x % kGroups, at = (int)blockIdx.x / kGroups;
    const int slab = at & ((1 << slab_bits) - 1), row0 = (at >> slab_bits) * 32;
    const int row = row0 + lane;  // bq * H + h
    const int d0 = slab * 64 + (kGroups == 1 ? slice * 8 : sub * 8 + slice * 32);
    const bool active = row < g.n_rows;
    const int bq = active ? g.H.div(row) : 0, h = active ? row - bq * a.H : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int np = 0, step = 1;            // partials of the row; float4 between its two pieces
    size_t stride = 0, mstride = 0;  // between partials: float4, (m, l)
    const float4 *src = nullptr;
    const float2 *ml = nullptr;
    if (!active) {
    } else if (g.plan.pairs > 0) {
        const int rt = row / kPrefixRows, rr = row % kPrefixRows, half_bits = slab_bits > 0 ? slab_bits + 5 : 6;
        const int2 meet = g.meet[rt];
        const size_t p0 = (size_t)meet.x + rt;
        np = meet.y;
        ml = g.ml + p0 * kPrefixRows + rr;
        // dim d0 of row rr: [rank][piece of 4 columns][lane half x 64 rows][4]
        const int hf = d0 >> half_bits, col = d0 & ((1 << half_bits) - 1), pieces = 1 << (half_bits - 2);
        src = reinterpret_cast<const float4 *>(g.part) + ((p0 * 2 + (rr >> 6)) * pieces + col / 4) * 128 + hf * 64 + (rr & 63);
        step = 128;
        stride = (size_t)pieces * 256;
        mstride = kPrefixRows;
    } else {
        np = a.splits;
        ml = a.part_ml + row;
        mstride = (size_t)g.n_rows;
        stride = (size_t)g.n_rows * a.D / 4;
        src = reinterpret_cast<const float4 *>(a.part_f + (size_t)bq * a.H * a.D);
        if (a.part_perm) {
            src += ((((size_t)(h >> 6) << slab_bits) + slab) * 1024) + ((h & 63) >> 4) * 256 + ((d0 & 31) / 4) * 32 + (h & 15) +
                   ((d0 >> 5) & 1) * 16;
            step = 32;
        } else {
            src += ((size_t)h * a.D + d0) / 4;
        }
    }
    // A few partials at a time, their (m, l) and rows all in flight together (a row without a key
    // was not written: whatever is there is not used), under a running maximum.
    float M = -INFINITY, L = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i0 = group; i0 < np; i0 += kAtOnce * kGroups) {
        float2 s[kAtOnce];
        float4 x[kAtOnce], y[kAtOnce];
        float top = M;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            s[i] = make_float2(-INFINITY, 0.f);
            if (i0 + i * kGroups < np) {
                s[i] = ml[(i0 + i * kGroups) * mstride];
                x[i] = src[(i0 + i * kGroups) * stride];
                y[i] = src[(i0 + i * kGroups) * stride + step];
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, s[i].x);
        const float f = M == top ? 1.f : exp2f(M - top);  // (also while both are -inf)
        M = top;
        L *= f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= f;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (s[i].x != -INFINITY) {
                const float w = exp2f(s[i].x - M);
                L = fmaf(w, s[i].y, L);
                acc[0] = fmaf(w, x[i].x, acc[0]); acc[1] = fmaf(w, x[i].y, acc[1]);
                acc[2] = fmaf(w, x[i].z, acc[2]); acc[3] = fmaf(w, x[i].w, acc[3]);
                acc[4] = fmaf(w, y[i].x, acc[4]); acc[5] = fmaf(w, y[i].y, acc[5]);
                acc[6] = fmaf(w, y[i].z, acc[6]); acc[7] = fmaf(w, y[i].w, acc[7]);
            }
    }
    if constexpr (kGroups > 1) {
        // group 0 adds up the others' in their order: [group - 1][slice][M, L, 8 sums][row]
        __shared__ float met[kGroups - 1][kSlices][10][32];
        if (group > 0) {
            met[group - 1][slice][0][lane] = M;
            met[group - 1][slice][1][lane] = L;
#pragma unroll
            for (int e = 0; e < 8; ++e) met[group - 1][slice][2 + e][lane] = acc[e];
        }
        __syncthreads();
        if (group == 0) {
            float top = M;
#pragma unroll
            for (int i = 0; i < kGroups - 1; ++i) top = fmaxf(top, met[i][slice][0][lane]);
            const float f = M == top ? 1.f : exp2f(M - top);
            M = top;
            L *= f;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] *= f;
#pragma unroll
            for (int i = 0; i < kGroups - 1; ++i) {
                const float m = met[i][slice][0][lane], w = m == -INFINITY ? 0.f : exp2f(m - M);
                L = fmaf(w, met[i][slice][1][lane], L);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, met[i][slice][2 + e][lane], acc[e]);
            }
        }
    }
    bool bad = false;
    if constexpr (kRedo) {
        // (the weights in L are the row's own: NaN that is in the sums alone may come from others' keys)
        const float sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
        bad = sum != sum && L == L && active && group == 0 && shares_row_tile(g, row);
    }
    if (a.sinks && active) L += exp2f(__ldg(a.sinks + h) * 1.4426950408889634f - M);
    const float inv = inverse_sum(M, L);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (group == 0) tile[lane][d0 % 64 + e] = acc[e] * inv;
    if constexpr (!kRedo) {
        __syncthreads();
    } else if (__syncthreads_or(bad)) {
        redo_rows(g, row, active, bad, d0, &tile[lane][d0 % 64]);
        __syncthreads();
    }
    // now a thread 8 dims of row threadIdx.x / 8, eight threads 128 contiguous bytes (with groups: two threads a row)
    const int r = (int)threadIdx.x / kSlices, c0 = kGroups == 1 ? (int)(threadIdx.x & 7) * 8 : sub * 8 + (int)(threadIdx.x & 1) * 32;
    if (r >= 32 || row0 + r >= g.n_rows) return;
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = tile[r][c0 + e];
    if (a.rope_cos && slab == (1 << slab_bits) - 1) {
        // conjugate rotation of the trailing 64 channels: channel D-64+j pairs with D-32+j
        const long long t = __ldg(a.q_pos + g.H.div(row0 + r));
        const bool first = c0 < 32;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 cs = rope_cs(a, t, (c0 & 31) + e);
            const float pv = tile[r][(c0 ^ 32) + e];
            o[e] = first ? o[e] * cs.x + pv * cs.y : o[e] * cs.x - pv * cs.y;
        }
    }
    *reinterpret_cast<uint4 *>(a.out + (size_t)(row0 + r) * a.D + slab * 64 + c0) = pack8(o);
}

// Which kernel a call takes, how it splits its keys, and where its partial rows lie in the workspace.
struct PagedPlan {
    PrefixPlan prefix;  // pairs > 0: attend_prefix.cu
    int splits;
    size_t keys, hi, lo, rq, part, ml, meet, bytes;  // offsets
};

size_t take(size_t &at, size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~size_t(255);
    return o;
}

// The most that a bf16 copy of an FP8 cache's rows may take; beyond it the gather kernel reads the codes in place.
constexpr long long kMaxCopyBytes = 1LL << 30;

// Estimated time in us of the two kernels, from a sweep (D 64..512, 8..128 heads, 1..64 queries, 0..16384
// shared and 64..4096 own entries): the gather kernel takes 2.6 us per tile of 64 keys and 64 heads of its
// busiest CTA (FP8: 5.6), attend_prefix.cu 0.9 to 1.45 us per unit and what its ranges' partials cost the merge.
// E.g. at D = 512, 128 heads: 8 requests over 1024 shared entries 22 us and 24 us, 32 over 1024 42 and 36,
// 32 over 16384 331 and 122; at D = 128, 16 heads: 16 over 1024 16 and 28, 64 over 16384 281 and 38.
// The host knows the tables' width, not the requests' lengths: `own` is what the width has room for.  The copy of an
// FP8 cache takes ~0.12 us per MiB on top (32 x 128 heads over 8192 entries, 192 own ones in tables of 192 / 16000:
// 77 and 141 us, 354 and 344 query by query); with that in the estimate too many calls of long requests go query
// by query (20 shapes where it decides: 1127 us in all with the rows together, 1258 without), so it stands without.
// The gather kernel reads a query's window; attend_prefix.cu goes through every row of the ring and clears those
// outside the window one by one, ~6 us per 128 of them (32 x 128 heads over 2048 entries, rings of 2048 / 8192
// rows: 59 / 59 us and 104 / 239; 64 x 16 heads over 4096: 92 / 92 and 120 / 366; 2 x 512 queries, 639 rows: 287 and 629).
bool prefix_pays(long long n_bq, int H, int D, long long n_shared, long long own, int nq, const PagedPlan &gather, int W,
                 int ring_rows, bool fp8, const PrefixPlan &pl) {
    const long long HH = (H + 63) / 64, keys = n_shared + own + W;
    const long long per = ((keys + 63) / 64 + gather.splits - 1) / gather.splits;
    const long long waves = (n_bq * HH * gather.splits + num_sms() - 1) / num_sms();
    const double t_gather = 8.0 + (gather.splits > 1 ? 2.0 : 0.0) + (fp8 ? 5.6 : 2.6) * (double)(waves * (per + 1));
    // requests whose rows a row tile holds
    const double requests = std::max(1.0, (double)kPrefixRows / ((double)H * nq));
    const double u = (double)((n_shared + kPrefixKeys - 1) / kPrefixKeys) + requests * (double)((own + W + 2 * kPrefixKeys - 17) / kPrefixKeys);
    const double units = u * pl.row_tiles, ranges = pl.ranges((int)std::min(units, 2e9));
    const double outside = requests * pl.row_tiles * (double)(ring_rows - W) / kPrefixKeys;
    const double unit = D == 512 ? 1.45 : (D == 256 ? 1.1 : 0.9);
    const double t_prefix = 14.0 + (fp8 ? 2.0 : 0.0) + unit * ((units + PrefixPlan::kPartCost * pl.row_tiles) / ranges) +
                            unit / 3 * (ranges / pl.row_tiles) + 6.0 * outside / ranges;
    return t_prefix < t_gather;
}

// rewrite: a gain, RoPE or a negative scale changes the query rows.  Either kernel keeps them in 16 bits, but the
// gather kernel at D = 512, where there is no room and they are rounded to 8: it is not taken for them if it need not.
PagedPlan paged_plan(int batch, int nq, int H, int D, int page, int max_pages, long long n_shared, int ring_rows, int W,
                     bool fp8, bool rewrite) {
    PagedPlan pl = {};
    const long long n_bq = (long long)batch * nq, rows = n_bq * H, cap = (long long)max_pages * page;
    const long long copy = fp8 ? (n_shared + batch * (cap - n_shared + ring_rows)) * D * (long long)sizeof(uint16_t) : 0;
    // units are counted in 32 bits, with what a row tile costs beside them: shared tiles and, of each request in a row
    // tile (one in part at either end), own ones
    const long long tiles = PrefixPlan::kPartCost + n_shared / kPrefixKeys + 1 +
                            (2 + kPrefixRows / H) * ((cap - n_shared + ring_rows) / kPrefixKeys + 2);
    size_t at = 0;
    pl.splits = attend_tc_plan(n_bq, H, cap + W);
    const PrefixPlan prefix = prefix_plan(std::min(rows, 0x7fffffffLL));
    if (rows <= 0x7fffffffLL - kPrefixRows && copy <= kMaxCopyBytes && tiles <= 0x7fffffffLL / (rows / kPrefixRows + 1) &&
        ((rewrite && D == 512) || prefix_pays(n_bq, H, D, n_shared, cap - n_shared, nq, pl, W, ring_rows, fp8, prefix))) {
        pl.prefix = prefix;
        if (rewrite) {
            pl.hi = take(at, (size_t)rows * D * sizeof(uint16_t));
            pl.lo = take(at, (size_t)rows * D * sizeof(uint16_t));
            pl.rq = take(at, (size_t)rows * sizeof(float));
        }
        if (fp8) pl.keys = take(at, (size_t)copy);
        pl.part = take(at, (size_t)pl.prefix.partials() * kPrefixRows * prefix_dims(D) * sizeof(float));
        pl.ml = take(at, (size_t)pl.prefix.partials() * kPrefixRows * sizeof(float2));
        pl.meet = take(at, (size_t)pl.prefix.row_tiles * sizeof(int2));
    } else if (pl.splits > 1) {
        pl.part = take(at, (size_t)pl.splits * rows * D * sizeof(float));
        pl.ml = take(at, (size_t)pl.splits * rows * sizeof(float2));
    }
    pl.bytes = at;
    return pl;
}

}  // namespace

size_t attend_paged_workspace_bytes(int batch, int nq, int H, int D, int page, int max_pages, long long n_shared,
                                    int ring_rows, int W, bool fp8, bool rewrite) {
    return paged_plan(batch, nq, H, D, page, max_pages, n_shared, ring_rows, W, fp8, rewrite).bytes;
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
    const PagedPlan pl =
        paged_plan(p.batch, a.nq, a.H, a.D, a.page, a.max_pages, p.n_shared, p.ring_rows, a.W, fp8, paged_rewrite(p));
    if (pl.bytes > 0 && (!ws || ws_bytes < pl.bytes)) return CSA_ERR_WORKSPACE;
    char *w = static_cast<char *>(ws);
    a.splits = pl.splits;
    MergeArgs g = {};
    g.a = a;
    g.H = FastDiv::by((uint32_t)a.H);
    g.n_rows = (int)(a.n_bq * a.H);
    int rc;
    if (pl.prefix.pairs > 0) {
        PrefixArgs x = {};
        x.a = a;
        x.plan = g.plan = pl.prefix;
        x.n_shared = p.n_shared;
        x.keys = p.pool;
        x.own_cap = fp8 ? (int)(a.N - p.n_shared) : -1;
        if (paged_rewrite(p)) {
            x.hi = reinterpret_cast<uint16_t *>(w + pl.hi);
            x.lo = reinterpret_cast<uint16_t *>(w + pl.lo);
            x.rq = reinterpret_cast<float *>(w + pl.rq);
            rc = launch_query_rows(x, st);
            if (rc != CSA_OK) return rc;
        }
        if (fp8) {
            uint16_t *keys = reinterpret_cast<uint16_t *>(w + pl.keys);
            rc = launch_expand_rows(x, keys, st);
            if (rc != CSA_OK) return rc;
            x.keys = keys;
        }
        g.part = x.part = reinterpret_cast<float *>(w + pl.part);
        g.ml = x.ml = reinterpret_cast<float2 *>(w + pl.ml);
        g.meet = x.meet = reinterpret_cast<int2 *>(w + pl.meet);
        g.keys = x.keys;
        g.n_shared = x.n_shared;
        g.own_cap = x.own_cap;
        g.hi = x.hi;
        g.lo = x.lo;
        g.rq = x.rq;
        rc = launch_attend_prefix(x, ctx, st);
        if (rc != CSA_OK) return rc;
    } else {
        if (pl.splits > 1) {
            a.part_f = reinterpret_cast<float *>(w + pl.part);
            a.part_ml = reinterpret_cast<float2 *>(w + pl.ml);
            a.part_perm = a.H % 64 == 0 ? 1 : 0;
        }
        rc = launch_attend_tc(a, ctx, st, false);
        if (rc != CSA_OK || pl.splits == 1) return rc;
        g.a = a;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.n_bq * a.H + 31) / 32 * (a.D / 64)));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    // partials of most rows: the splits, or the ranges of a row tile and one that both its ends share
    const int partials = pl.prefix.pairs > 0 ? pl.prefix.pairs / pl.prefix.row_tiles + 1 : pl.splits;
    // groups while their blocks leave SMs idle: 32 rows x 64 dims of 74 partials 12.5 -> 10.4 us (the whole call),
    // 256 x 256 of 37 23.4 -> 20.5; but 512 x 512 of some ten 26.7 -> 28.7, 1536 x 128 41.6 -> 43.1
    const bool groups = partials > 6 && 2 * cfg.gridDim.x <= (unsigned)num_sms();
    if (groups) cfg.gridDim.x *= 4;
    // (128 heads: a row tile is one query's.  Without the second look 32 x 128 rows take 1 us less)
    const bool redo = pl.prefix.pairs > 0 && a.H < kPrefixRows;
    const auto launch = [&](auto kernel, auto kernel_redo) { return cudaLaunchKernelEx(&cfg, redo ? kernel_redo : kernel, g); };
    const cudaError_t e = groups         ? launch(attend_merge_kernel<4, 4, false>, attend_merge_kernel<4, 4, true>)
                          : partials <= 4 ? launch(attend_merge_kernel<2, 1, false>, attend_merge_kernel<2, 1, true>)
                                          : launch(attend_merge_kernel<6, 1, false>, attend_merge_kernel<6, 1, true>);
    return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // namespace csa
