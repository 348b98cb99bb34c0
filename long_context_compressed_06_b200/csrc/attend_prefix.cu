// attend_prefix.cu -- hca_attend_paged for a batch whose requests share a long
// prefix: the query rows of the whole batch as one product with the shared
// entries, and each request's own entries and window beside it.
//
// With the query rows of every request stacked, Q is [R = batch * nq * H][D]
// and the shared entries X [n_shared][D] are keys and values of all of them:
//   S = scale / RMS(q) * Q X^T,   P = exp2(S - m),   O = P X
// with the running maximum m and sum l of every row kept per tile of 128 keys
// (m raised only when it grows by more than 2^8, so that O in tensor memory is
// rarely rescaled).  A tile of 128 rows continues with the own keys of each of
// its requests, 128 at a time, the rows of other requests masked: with H = 128
// heads a row tile is one request and nothing is wasted, and a batch of small
// heads shares the tile's tensor work that the mask throws away.  (Masked rows have
// weights of 0; what 0 times a key that is not finite does to them the merge finds
// and mends, attend_paged.cu.)  O, m and l of
// a range of tiles go out in 32 bits and are merged (attend_paged.cu).
//
// A pair of SMs owns 128 rows (cta_group::2, M = 128): every MMA reads half of
// its B operand from each SM, and an accumulator takes 64 rows x N/2 columns x
// two lane halves of each SM's tensor memory, so that O at D = 512 fits in 256
// columns beside two S buffers.  One SM alone would have to run at M = 64, half
// the tensor rate (128 rows x 512 fp32 columns fill its tensor memory).
// Column c of lane half f of O is dim f * DP / 2 + c.
// The price is that each SM loads 64 of a tile's 128 keys whole (its half of
// K's rows) and all 128 keys by half their dims (its half of V's columns):
// 128 KiB per SM and tile at D = 512, 1.33 times what one copy would be.
// At D = 512 a tile takes ~3200 cycles, two thirds of them MMAs (QK 1056 + P.V
// 1056); 32 row tiles of 8064 + 192 keys take 64 us with the merge.  Nothing is at
// its limit there (tensor pipe 51 %, L2 34 %; a copy of the kernel that loaded half
// of V took as long): it is bound by the roles' waits for one another and for their
// instructions (1.9 warps of a quarter SM wait for one at every issue).
// At D = 128 the softmax bounds it: ~1850 cycles a tile, a third of it exponentials.
//
// A gain, RoPE or a negative scale changes the query rows first, and rounding
// them to bf16 again would cost as much accuracy as the output's own rounding
// does (16 x 4 queries of 128 heads over 4096 entries, norm of the error against 64
// bits by that of the output: 2.49e-3 instead of 1.85e-3, of which the output's
// rounding is 1.66e-3).  A launch before
// writes them as a sum of two bf16 numbers (hi + lo, 16 bits), and S gets both
// products; lo passes through K's ring beside each piece of K, since at D = 512
// shared memory has no room for it (64 queries x 128 heads over 4096 entries 74 ->
// 105 us: half more products and half more loads).
//
// Warps: 0 and 1 producers of K, 2 and 3 of V, 4 and 5 MMA issuers of Q K^T and of
// P V on the pair's leader (one thread for both was busy for longer than the
// tensor cores: a satisfied barrier wait takes ~140 cycles, an MMA ~20), 6
// tensor memory and the query tiles, 7 the planner, 8..15 softmax: two groups of
// four warps take the tiles in turn, two threads per row (64 keys each), so that
// the waits and exchanges of one tile overlap the exponentials of the next (all
// eight warps on one tile took ~2500 cycles a tile, most of it latency).
// The planner walks the pair's tiles a few ahead of everyone, describes each in
// shared memory (struct Tile) and brings own rows into L2 (the producers are one
// tile ahead at D = 512).  Each role's code is kept small on purpose: unrolled
// loops that run once per row tile, or between waits, cost more in instruction
// misses than in work (rolled, 32 x 128 heads over 8064 entries 64.8 -> 63.8 us,
// 96 x 16 heads over 16384 43.9 -> 42.1).
// K and V have a ring of 16 KiB slots each; every tile passes through both, and
// two producer warps take a ring's positions in turn.  Rows arrive by TMA,
// entries in boxes that never cross a page, window rows 16 at a time in the
// order of the ring; FP8 rows are expanded to a bf16 copy by a launch before
// (expanding them in the producers took ~12K cycles a tile).  (A slot's phase
// bit tells its use from the one before only: whoever waits on a ring passes
// every use.)
//
// The tiles of all row tiles ("units") are counted on the device from the
// positions and dealt to the pairs in balanced contiguous ranges.
#include <algorithm>
#include <cstring>

#include "attend_common.cuh"
#include "common.cuh"
#include "kernels.h"
#include "quant_fp8.cuh"
#include "tc.cuh"

namespace csa {
namespace {

constexpr int kThreads = 512;
constexpr int kProducers = 4, kQkWarp = 4, kPvWarp = 5, kQueryWarp = 6, kPlanWarp = 7, kSoftWarp0 = 8, kSoftWarps = 8;
constexpr int kSlots = 4;  // of each ring
constexpr uint32_t kSlotBytes = 16384;  // K: 64 keys x 128 dims, V: 16384 / DP keys x DP / 2 dims
constexpr uint32_t kPBytes = 16384;     // 64 rows x 128 keys, bf16
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t kSCols = 256;        // first column of the S buffers (64 columns each)
constexpr int kSBufs = 4;

template <int DP>
struct Layout {
    static constexpr int kPieces = DP / 128;              // slots of a K tile, and of a V tile, per SM
    static constexpr int kPvN = DP < 256 ? DP : 256;      // N of one P.V MMA
    static constexpr int kPvMmas = DP / kPvN;             // MMAs per 16 keys
    static constexpr int kVKeys = 16384 / DP;             // keys of a V slot
    static constexpr int kVChunks = DP / 128;             // its 64-dim chunks (this SM's half of V's columns)
    static constexpr int kDescs = DP < 512 ? 16 : 8;      // tiles described ahead (8: what shared memory is left)
    static constexpr uint32_t kQBytes = 64 * DP * 2;      // [DP/64][64 rows][128 B]
};

struct Params {
    AttendArgs a;
    PrefixPlan plan;
    int n_shared;
    int linear;
    int lo;           // the query rows are hi + lo, and rq holds their factors
    int dependent;    // launched as a programmatic dependent of what writes the copies
    const float *rq;
    int2 *meet;       // [row_tiles], see PrefixArgs
    FastDiv H, nq, m, page, ring;
    int batch;
    int own_cap;           // linear: rows of the copy for one request's own entries
    int box;          // entries that one copy brings at most (none crosses a page): 16, 32 or 64
    int vbox;         // those of a V copy: at most one slot's
    float *part;
    float2 *ml;
    uint32_t idesc_qk, idesc_pv;
    DevCtx ctx;
};

// One tile of 128 keys, as the planner describes it.
enum : int { kShared = 1, kFirst = 2, kLast = 4, kEnd = 8, kMixed = 16, kMissingShift = 8, kRingShift = 16 };
struct Tile {
    int flags;         // kShared: entries of all requests, else own keys of request b; kFirst / kLast of a pair's
                       // part of a row tile; kEnd: no tile; kMixed: window rows among the keys.  Of keys 16 i ..
                       // 16 i + 15, bit kMissingShift + i: entries without a page, kRingShift + i: window rows
    int ent_rt;        // keys [0, ent) are entries that some row sees; the row tile: ent | rt << 8
    int n;             // kFirst: tiles of the part
    int b;
    int e_first;       // entry index of key 0
    int r_first;       // ring row of key 0 (kMixed: keys from -r_first on, where that is positive)
    int rows[8];       // row of key 16 i in the pool, the rings or (linear) the copy; < 0: none, reads as zeros
    uint32_t zero[4];  // keys that a copy brings and no row takes: cleared in V
    CSA_DEVINL int ent() const { return ent_rt & 255; }
    CSA_DEVINL int rt() const { return (int)((uint32_t)ent_rt >> 8); }
};

struct Smem {
    uint8_t *q, *slots, *p;  // slots: K's ring, then V's; so are their barriers
    uint64_t *full, *empty, *sfull, *sempty, *pfull, *pvdone, *qland, *qready, *qempty, *vfix, *dfull, *dempty, *rbar;
    Tile *desc;  // [kDescs]
    // [2 x 32 rows][tile parity][2 halves of the keys][32] the row's maximum and the tile's tag in one word (tagged)
    uint32_t *xch;
    uint32_t *tmem_slot;
    int *abort_flag;
};

template <int DP>
CSA_DEVINL Smem carve(uint8_t *raw) {
    Smem s;
    s.q = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    s.slots = s.q + Layout<DP>::kQBytes;
    s.p = s.slots + 2 * kSlots * kSlotBytes;
    s.xch = reinterpret_cast<uint32_t *>(s.p + 2 * kPBytes);
    s.desc = reinterpret_cast<Tile *>(s.xch + 256);
    uint64_t *bars = reinterpret_cast<uint64_t *>(s.desc + Layout<DP>::kDescs);
    s.full = bars;
    s.empty = s.full + 2 * kSlots;
    s.dfull = s.empty + 2 * kSlots;
    s.dempty = s.dfull + Layout<DP>::kDescs;
    s.sfull = s.dempty + Layout<DP>::kDescs;
    s.sempty = s.sfull + kSBufs;
    s.pfull = s.sempty + kSBufs;
    s.pvdone = s.pfull + 2;
    s.rbar = s.pvdone + 2;  // [2 x 32 rows]
    s.qland = s.rbar + 2;
    s.qready = s.qland + 1;
    s.qempty = s.qready + 1;
    s.vfix = s.qempty + 1;  // [2]
    s.tmem_slot = reinterpret_cast<uint32_t *>(s.vfix + 2);
    s.abort_flag = reinterpret_cast<int *>(s.tmem_slot + 1);
    return s;
}

template <int DP>
constexpr size_t smem_bytes() {
    return 1024 + Layout<DP>::kQBytes + 2 * kSlots * kSlotBytes + 2 * kPBytes + 1024 + Layout<DP>::kDescs * sizeof(Tile) +
           (4 * kSlots + 2 * Layout<DP>::kDescs + 2 * kSBufs + 11) * 8 + 8;
}
static_assert(smem_bytes<512>() <= 227 * 1024, "shared memory of one CTA");

// ---------------------------------------------------------------- units
// The tiles of row tile rt, in order: the shared entries that any of its rows
// sees, then request by request the own keys of its queries in the row tile.
CSA_DEVINL int visible(const Params &p, int t, int cap) {  // min((t + 1) / m, cap)
    if (t < 0) return 0;
    const int q = p.m.div(t), v = q + (t - q * (int)p.m.d == (int)p.m.d - 1 ? 1 : 0);
    return v < cap ? v : cap;
}

// The own keys of queries [q0, q1] of one request: entries n_shared..n_shared + n_own - 1,
// then, from a multiple of 16 on, the rows of its ring in order.
struct Own {
    int n_own;
    uint32_t total;  // with the entries padded to 16 and every row of the ring (no live query: 0)
    CSA_DEVINL uint32_t ring0() const { return ((uint32_t)n_own + 15u) & ~15u; }  // key of ring row 0
    CSA_DEVINL int tiles() const { return (int)((total + (uint32_t)kPrefixKeys - 1u) / (uint32_t)kPrefixKeys); }
};

CSA_DEVINL Own own_keys(const Params &p, int q0, int q1) {
    int vis = 0, t1 = -1;
#pragma unroll 1
    for (int q = q0; q <= q1; ++q) {
        const int t = __ldg(p.a.q_pos + q);
        vis = std::max(vis, visible(p, t, (int)p.a.N));
        t1 = std::max(t1, t);
    }
    Own o;
    o.n_own = std::max(0, vis - p.n_shared);
    o.total = t1 < 0 ? 0u : o.ring0() + (uint32_t)p.a.win_rows;
    return o;
}

// Queries (rows of q_pos) bq0..bq1 of row tile rt.
struct Queries {
    int bq0, bq1;
};

CSA_DEVINL Queries queries_of(const Params &p, int rt) {
    Queries r;
    const int row0 = rt * kPrefixRows;
    r.bq0 = p.H.div(row0);
    r.bq1 = std::min((int)p.a.n_bq - 1, p.H.div(row0 + kPrefixRows - 1));
    return r;
}

// Units of row tile rt (x) and how many shared entries its rows see (y), by `subs`
// consecutive lanes that share its requests (every lane has both); rt past the last: 0.
CSA_DEVINL int2 count_units(const Params &p, int rt, int subs) {
    int vmax = 0, n = 0;
    if (rt < p.plan.row_tiles) {
        const Queries r = queries_of(p, rt);
        const int b1 = p.nq.div(r.bq1);
#pragma unroll 1
        for (int b = p.nq.div(r.bq0) + (threadIdx.x & (subs - 1)); b <= b1; b += subs) {
            const int q0 = std::max(r.bq0, b * p.a.nq), q1 = std::min(r.bq1, b * p.a.nq + p.a.nq - 1);
            n += own_keys(p, q0, q1).tiles();
#pragma unroll 1
            for (int q = q0; q <= q1; ++q) vmax = std::max(vmax, visible(p, __ldg(p.a.q_pos + q), p.n_shared));
        }
    }
#pragma unroll 1
    for (int d = 1; d < subs; d <<= 1) {
        n += __shfl_xor_sync(0xffffffffu, n, d);
        vmax = std::max(vmax, __shfl_xor_sync(0xffffffffu, vmax, d));
    }
    return make_int2(n + (vmax + kPrefixKeys - 1) / kPrefixKeys, vmax);
}

// A pair's units: `left` of them from number x of row tile rt on, whose counts are n.
struct Units {
    int left, rt, x;
    int2 n;
};

// Units of the row tiles, by the whole block, to `counts` (at most kCounts of them).
constexpr int kCounts = (int)(2 * kPBytes / sizeof(int2));

CSA_DEVINL int count_lanes(const Params &p) {  // lanes per row tile: about its requests
    int subs = 1;
    while (subs < 32 && subs * p.a.H * p.a.nq < kPrefixRows) subs *= 2;
    return subs;
}

CSA_DEVINL void count_all(const Params &p, int2 *counts) {
    const int subs = count_lanes(p), RT = std::min(p.plan.row_tiles, +kCounts), step = kThreads / subs;
#pragma unroll 1
    for (int r0 = 0; r0 < RT; r0 += step) {
        const int rt = r0 + (int)threadIdx.x / subs;
        const int2 n = count_units(p, rt, subs);
        if (rt < RT && (threadIdx.x & (subs - 1)) == 0) counts[rt] = n;
    }
}

// By one warp; `write`: also the ranges of every row tile.
CSA_DEVINL Units deal_units(const Params &p, const int2 *counts, int pair, bool write) {
    const int lane = threadIdx.x & 31, RT = p.plan.row_tiles, subs = count_lanes(p);
    int total = 0, units = 0, cost = 0, inc = 0;
    int2 n = {0, 0};
    const auto pass = [&](int r0) {  // n: counts of row tile r0 + lane; its cost; inc: costs up to it in this pass
        n = make_int2(0, 0);
        if (r0 + 32 <= kCounts) {
            if (r0 + lane < RT) n = counts[r0 + lane];
        } else {
#pragma unroll 1
            for (int l0 = 0; l0 < 32; l0 += 32 / subs) {
                const int2 c = count_units(p, r0 + l0 + lane / subs, subs);
                const int from = (lane - l0) * subs & 31, x = __shfl_sync(0xffffffffu, c.x, from), y = __shfl_sync(0xffffffffu, c.y, from);
                if (lane >= l0 && lane < l0 + 32 / subs) n = make_int2(x, y);
            }
        }
        cost = n.x > 0 ? n.x + PrefixPlan::kPartCost : 0;
        inc = cost;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += up;
        }
    };
#pragma unroll 1
    for (int r0 = 0; r0 < RT; r0 += 32) {
        pass(r0);
        const int sum = __shfl_sync(0xffffffffu, inc, 31);
        total += sum;
        units += sum - PrefixPlan::kPartCost * __popc(__ballot_sync(0xffffffffu, cost > 0));
    }
    const int ranges = p.plan.ranges(units);
    // for the merge: which ranges meet each row tile
    if (write) {
        int base = 0;
#pragma unroll 1
        for (int r0 = 0; r0 < RT; r0 += 32) {
            if (RT > 32) pass(r0);
            const int at = base + inc - cost;
            if (r0 + lane < RT) {
                const int q0 = cost > 0 ? range_of(at + PrefixPlan::kPartCost, ranges, total) : 0;
                p.meet[r0 + lane] = make_int2(q0, cost > 0 ? range_of(at + cost - 1, ranges, total) - q0 + 1 : 0);
            }
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    Units u = {0, 0, 0, {0, 0}};
    if (total == 0 || pair >= ranges) return u;
    // the units between two places among all costs
    const int u0 = range_begin(pair, ranges, total), u1 = range_begin(pair + 1, ranges, total);
#pragma unroll 1
    for (int r0 = 0, base = 0; r0 < RT && base < u1; r0 += 32) {
        if (RT > 32) pass(r0);
        const int start = base + inc - cost;
        const int c0 = std::min(std::max(u0 - start - PrefixPlan::kPartCost, 0), n.x);  // its units before u0, u1
        const int c1 = std::min(std::max(u1 - start - PrefixPlan::kPartCost, 0), n.x);
        u.left += __reduce_add_sync(0xffffffffu, c1 - c0);
        const uint32_t here = __ballot_sync(0xffffffffu, start <= u0 && u0 < start + cost);
        if (here) {
            const int l = __ffs(here) - 1;
            u.rt = r0 + l;
            u.x = __shfl_sync(0xffffffffu, c0, l);
            u.n = make_int2(__shfl_sync(0xffffffffu, n.x, l), __shfl_sync(0xffffffffu, n.y, l));
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    return u;
}

// mbar_wait (common.cuh) with the hardware's own wait made long and the rest out of line: some thirty waits
// inlined, polled by a dozen idle warps, cost the working warps their instruction fetch.
CSA_DEVINL bool try_wait_long(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(100000u)  // ns
        : "memory");
    return ok != 0;
}

__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, const DevCtx &ctx, volatile int *abort) {
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (try_wait_long(bar, parity)) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > ctx.budget_ns) {
            record_status(ctx.status, CSA_ERR_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
}

CSA_DEVINL bool bar_wait(uint32_t bar, uint32_t parity, const DevCtx &ctx, volatile int *abort) {
    return try_wait_long(bar, parity) || wait_on(bar, parity, ctx, abort);
}

CSA_DEVINL bool warp_wait(uint32_t bar, uint32_t parity, const DevCtx &ctx, volatile int *abort) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, ctx, abort));
}

// Where a few warps meet (an mbarrier of one arrival per warp, `uses` its phases so far): a named
// barrier is cheaper, but would hang for good if a warp had given up a wait and left.
CSA_DEVINL bool warps_meet(uint32_t bar, uint32_t &uses, const DevCtx &ctx, volatile int *abort) {
    __syncwarp();
    mbar_arrive(bar, (threadIdx.x & 31) == 0);
    return warp_wait(bar, uses++ & 1u, ctx, abort);
}

// The tile's query rows as they landed: this thread's quarter of row r (units
// q4, q4 + 4, .. of 8 dims) -> its sum of squares (of an infinite element: NaN, as its normalised row is).
template <int DP>
CSA_DEVINL uint4 *query_unit(uint8_t *q, int r, int unit) {
    return reinterpret_cast<uint4 *>(q + (unit >> 3) * 8192 + r * 128 + (((unit & 7) ^ (r & 7)) << 4));
}

template <int DP>
CSA_DEVINL float query_squares(uint8_t *q, int r, int q4) {
    float ss[2] = {0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < DP / 32; ++i) {
        float x[8];
        unpack8(*query_unit<DP>(q, r, q4 + 4 * i), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[e & 1] = fmaf(x[e], x[e], ss[e & 1]);
    }
    float sum = ss[0] + ss[1];
    if (sum == INFINITY)  // or only too large for 32 bits
#pragma unroll 1
        for (int i = 0; i < DP / 32; ++i) {
            float x[8];
            unpack8(*query_unit<DP>(q, r, q4 + 4 * i), x);
            for (int e = 0; e < 8; ++e) sum = fmaf(x[e], 0.f, sum);
        }
    return sum;
}

// 1 / RMS of a row of these squares times the softmax scale (its sign is the query
// rows'), in log2 units; above 0, so that a masked score stays -inf (a NaN stays one)
CSA_DEVINL float row_factor(const AttendArgs &a, float ss) {
    const float f = (1.0f / sqrtf(ss / (float)a.D + a.eps)) * fabsf(a.scale) * 1.4426950408889634f;
    return f < 1e-37f ? 1e-37f : f;
}

// A row's maximum is exchanged without its last kTagBits bits (rounded towards zero by up to 3 steps of 32
// bits), where the tile's tag goes: a word's reader finds what it waits for or the word's use before.
constexpr uint32_t kTagBits = 2, kTagMask = (1u << kTagBits) - 1u;
CSA_DEVINL uint32_t tag_of(uint32_t g) { return (g >> 1) & kTagMask; }  // (a word serves every other tile)
CSA_DEVINL float untagged(uint32_t x) { return __uint_as_float(x & ~kTagMask); }
CSA_DEVINL uint32_t tagged(float v, uint32_t g) { return (__float_as_uint(v) & ~kTagMask) | tag_of(g); }
// Those 3 steps are 48 log2 units below 2^28, and the weights' range has room for them.  From 2^28 on (where a
// score's own rounding is 16 units and more) they would overflow, or be 0 under a negative maximum: there the
// differences between scores and maximum are scaled so that a step is 16 units, and a key one step away weighs
// 2^-16.  The factor of a maximum m: a power of two, 1 below 2^28.
CSA_DEVINL float difference_scale(float m) {
    const int over = (int)((__float_as_uint(m) >> 23) & 255u) - (127 + 27);
    return __uint_as_float((uint32_t)(127 - std::max(over, 0)) << 23);
}

// the first n of 32 bits
CSA_DEVINL uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u); }

// bits x..y (either may lie outside)
CSA_DEVINL uint32_t bits_between(int x, int y) { return low_bits(y + 1) & ~low_bits(x); }

// The ring rows that hold the window of a query: w0..w1, or (w0 > w1) ..w1 and w0.. .
struct Window {
    int w0, w1;
};

CSA_DEVINL Window window_of(const Params &p, int t) {  // t >= 0
    return {p.ring.mod(std::max(0, t - p.a.W + 1)), p.ring.mod(t)};
}

// which of ring rows k0..k0 + 31 they are
CSA_DEVINL uint32_t ring_bits(const Params &p, const Window &w, int k0) {
    return w.w0 <= w.w1 ? bits_between(w.w0 - k0, w.w1 - k0)
                        : bits_between(-k0, w.w1 - k0) | bits_between(w.w0 - k0, (int)p.ring.d - 1 - k0);
}

// The row of a query at t, of request b, that sees vis entries.
struct Row {
    int t, vis, b;
    Window w;
};

// Which of keys off..off + 31 of a tile it takes.
CSA_DEVINL uint32_t key_mask(const Params &p, const Tile &d, int off, const Row &r) {
    const int flags = d.flags;
    if (!(flags & kShared) && r.b != d.b) return 0u;
    uint32_t mask = low_bits(std::min(r.vis - d.e_first, d.ent()) - off);
    const int miss = flags >> (kMissingShift + off / 16);
    mask &= ~((miss & 1 ? 0x0000ffffu : 0u) | (miss & 2 ? 0xffff0000u : 0u));
    if ((flags & kMixed) && r.t >= 0) mask |= ring_bits(p, r.w, d.r_first + off);
    return mask;
}

// The tensor maps of one call, [64-dim chunk][row][64] each.
struct Maps {
    CUtensorMap q, lo;     // 64 rows x 2 chunks
    CUtensorMap k, v;      // pool or copy: box rows x 2 chunks (box 64) or 1, vbox rows x an SM's half of V
    CUtensorMap k16, v16;  // pool, 16 rows x 1 chunk, 16 rows x an SM's half
    CUtensorMap rk16, rv16;  // the rings, the same
};

template <int DP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attend_prefix_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    using Lt = Layout<DP>;
    constexpr uint32_t kDescs = Lt::kDescs;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const Smem s = carve<DP>(smem_raw);
    const AttendArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_rank(), pair = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kSlots; ++i) {
            mbar_init(s.full + i, 2);   // used on the leader: each CTA's producer (+ bytes of both)
            mbar_init(s.empty + i, 1);  // commit
        }
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(s.sfull + i, 1);
            mbar_init(s.sempty + i, kSoftWarps);  // leader: a group's warps in both CTAs
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s.pfull + i, kSoftWarps);  // leader: the same
            mbar_init(s.pvdone + i, 1);
            mbar_init(s.rbar + i, kSoftWarps / 2);
        }
        mbar_init(s.qland, 1);
        mbar_init(s.qready, 2);  // leader: each CTA's query warp
        mbar_init(s.qempty, 1 + kSoftWarps);
        for (int i = 0; i < 2; ++i) mbar_init(s.vfix + i, 1);
        for (int i = 0; i < kDescs; ++i) {
            mbar_init(s.dfull + i, 1);
            mbar_init(s.dempty + i, kSoftWarps / 2 + (rank == 0 ? 1 : 2));  // a group, the query tiles', the prefetching warp
        }
        *s.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kQueryWarp) tc::tmem_alloc_2sm(smem_u32(s.tmem_slot), 512);
    __syncwarp();
    // Both CTAs' barriers and tensor memory exist past the wait.  (An arrival waits for what its warp has
    // on the way to memory: it comes before the counts.)
    tc::cluster_arrive();
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&maps.q);
        tc::prefetch_tmap(&maps.k);
        tc::prefetch_tmap(&maps.v);
    }
    if (threadIdx.x < 256) s.xch[threadIdx.x] = kTagMask;  // not tile 0's or 1's
    count_all(p, reinterpret_cast<int2 *>(s.p));  // (P is written long after the planner has read them)
    tc::fence_before_sync();
    __syncthreads();
    if (warp != kPlanWarp) tc::cluster_wait();  // (the planner's barriers are its own CTA's)
    tc::fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = *s.tmem_slot;

    // tile number g's description, once it is there (null: given up)
    const auto desc_of = [&](uint32_t g) -> const Tile * {
        return bar_wait(smem_u32(s.dfull + g % kDescs), (g / kDescs) & 1u, p.ctx, s.abort_flag) ? s.desc + g % kDescs
                                                                                                 : nullptr;
    };
    const auto warp_desc_of = [&](uint32_t g) -> const Tile * {
        const Tile *d = desc_of(g);
        return __all_sync(0xffffffffu, d != nullptr) ? d : nullptr;
    };
    bool copies = false;  // given up with TMA copies in flight, maybe

    if (warp < kProducers) {
        // ------------------------------------------------------------ producers
        // TMA copies are issued by one thread inside an elect_one branch (one issued by every lane
        // under a guard, or by a diverged lane, took ~200 cycles: more than the MMAs that it feeds).
        if (p.dependent) asm volatile("griddepcontrol.wait;" ::: "memory");
        const bool v = warp >= 2;  // K's or V's ring
        const int ring = v ? kSlots : 0;
        const uint32_t full0 = tc::map_to_rank(smem_u32(s.full + ring), 0), slots = smem_u32(s.slots) + ring * kSlotBytes;
        const uint32_t vfix = smem_u32(s.vfix + (warp & 1));
        uint32_t it = 0, nfix = 0;  // ring position
        bool ok = true;
        for (uint32_t g = 0; ok; ++g) {
            const Tile *dp = warp_desc_of(g);
            if (!(ok = dp != nullptr)) break;
            const Tile &d = *dp;
            if (d.flags & kEnd) break;
            const int lo = v ? 0 : p.lo;  // K's ring: a piece of K, (lo) the query rows' piece beside it
#pragma unroll 1
            for (int x = 0; x < Lt::kPieces << lo && ok; ++x, ++it) {
                if ((it ^ (uint32_t)warp) & 1u) continue;
                const int w = x >> lo;
                const uint32_t sl = it % kSlots, par = ((it / kSlots) & 1u) ^ 1u, empty = smem_u32(s.empty + ring + sl);
                const uint32_t dst = slots + sl * kSlotBytes, full = full0 + sl * 8;
                if (!(ok = warp_wait(empty, par, p.ctx, s.abort_flag))) break;
                const bool mixed = d.flags & kMixed;
                const int vbox = mixed ? 16 : p.vbox;
                if (!v) {
                    if (tc::elect_one()) {
                        mbar_arrive_expect_tx_cluster(full, kSlotBytes);
                        if (lo && (x & 1)) {
                            tc::tma_load_3d_2sm(dst, &maps.lo, full, 0, d.rt() * kPrefixRows + rank * 64, 2 * w);
                        } else if (p.box == 64 && !mixed) {
                            tc::tma_load_3d_2sm(dst, &maps.k, full, 0, d.rows[rank * 4], 2 * w);
                        } else {
                            const int box = mixed ? 16 : p.box;
#pragma unroll 1
                            for (int y = 0; y < 64; y += box) {
                                const int i = rank * 4 + y / 16, row = d.rows[i];
                                const CUtensorMap *map =
                                    !mixed ? &maps.k : (d.flags >> (kRingShift + i)) & 1 ? &maps.rk16 : &maps.k16;
                                tc::tma_load_3d_2sm(dst + y * 128, map, full, 0, row, 2 * w);
                                tc::tma_load_3d_2sm(dst + 8192 + y * 128, map, full, 0, row, 2 * w + 1);
                            }
                        }
                    }
                    __syncwarp();
                    continue;
                }
                // V: keys that no row takes have zero weights; their values (anything, in memory) are
                // cleared where a copy brings them
                bool fix = false;
#pragma unroll
                for (int i = 0; i < Lt::kVKeys / 32; ++i) fix |= d.zero[w * (Lt::kVKeys / 32) + i] != 0u;
                if (tc::elect_one()) {
                    const uint32_t bar = fix ? tc::map_to_rank(vfix, rank) : full;
                    mbar_arrive_expect_tx_cluster(bar, kSlotBytes);
#pragma unroll 1
                    for (int y = 0; y < Lt::kVKeys; y += vbox) {
                        const int i = (w * Lt::kVKeys + y) / 16;
                        const CUtensorMap *map =
                            !mixed ? &maps.v : (d.flags >> (kRingShift + i)) & 1 ? &maps.rv16 : &maps.v16;
                        tc::tma_load_3d_2sm(dst + y * (Lt::kVChunks * 128), map, bar, 0, d.rows[i], rank * Lt::kVChunks);
                    }
                }
                __syncwarp();
                if (fix) {
                    if (!(ok = warp_wait(vfix, nfix & 1u, p.ctx, s.abort_flag))) break;
                    ++nfix;
                    // key e of the slot, chunk c: [e / vbox][c][e % vbox][128 B]
                    const int vsh = 31 - __clz(vbox);
#pragma unroll 1
                    for (int i = 0; i < Lt::kVKeys / 32; ++i)
#pragma unroll 1
                        for (uint32_t z = d.zero[w * (Lt::kVKeys / 32) + i]; z; z &= z - 1) {
                            const int e = i * 32 + __ffs(z) - 1;
                            const uint32_t line = ((((uint32_t)(e >> vsh) * Lt::kVChunks + (lane >> 3)) << vsh) + (e & (vbox - 1)));
                            if (lane < Lt::kVChunks * 8)
                                *reinterpret_cast<uint4 *>(s.slots + (ring + sl) * kSlotBytes + line * 128 + (lane & 7) * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    mbar_arrive_cluster(full, lane == 0);
                }
            }
        }
        copies = !ok;
    } else if (warp == kQkWarp) {
        // ------------------------------------------------------------ Q K^T (one thread of the leader)
        if (rank == 0 && tc::elect_one()) {
            const uint64_t qdesc = tc::smem_desc(smem_u32(s.q), 1024, tc::kLayoutSw128);
            const uint64_t kdesc = tc::smem_desc(smem_u32(s.slots), 1024, tc::kLayoutSw128);
            uint32_t nq = 0, it = 0;
            bool ok = true;
            for (uint32_t g = 0; ok; ++g) {
                const Tile *d = desc_of(g);
                if (!d) break;
                const int flags = d->flags;
                if (flags & kEnd) break;
                const uint32_t b = g % kSBufs;
                if (flags & kFirst) {
                    if (!bar_wait(smem_u32(s.qready), nq & 1u, p.ctx, s.abort_flag)) break;
                    ++nq;
                }
                if (!bar_wait(smem_u32(s.sempty + b), ((g / kSBufs) & 1u) ^ 1u, p.ctx, s.abort_flag)) break;
#pragma unroll 1
                for (int w = 0; w < Lt::kPieces; ++w, ++it) {
                    const uint32_t sl = it % kSlots;
                    if (!(ok = bar_wait(smem_u32(s.full + sl), (it / kSlots) & 1u, p.ctx, s.abort_flag))) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // 16 dims each: chunk 2 w + k / 4
                        const uint32_t off = (k >> 2) * 8192 + (k & 3) * 32;
                        tc::mma_f16_2sm(tmem + kSCols + b * 64, qdesc + ((w * 16384 + off) >> 4),
                                        kdesc + ((sl * kSlotBytes + off) >> 4), p.idesc_qk, (w | k) ? 1u : 0u);
                    }
                    if (p.lo) {
                        ++it;
                        const uint32_t ll = it % kSlots;
                        if (!(ok = bar_wait(smem_u32(s.full + ll), (it / kSlots) & 1u, p.ctx, s.abort_flag))) break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t off = (k >> 2) * 8192 + (k & 3) * 32;
                            tc::mma_f16_2sm(tmem + kSCols + b * 64, kdesc + ((ll * kSlotBytes + off) >> 4),
                                            kdesc + ((sl * kSlotBytes + off) >> 4), p.idesc_qk, 1u);
                        }
                        tc::mma_commit_2sm(smem_u32(s.empty + ll));
                    }
                    tc::mma_commit_2sm(smem_u32(s.empty + sl));
                }
                if (!ok) break;
                tc::mma_commit_2sm(smem_u32(s.sfull + b));
                if (flags & kLast) tc::mma_commit_2sm(smem_u32(s.qempty));
            }
        }
    } else if (warp == kPvWarp) {
        // ------------------------------------------------------------ P V (one thread of the leader)
        if (rank == 0 && tc::elect_one()) {
            // V as stored, [keys][dims] (MN-major): 64-dim chunks vbox * 128 bytes apart, 8-key groups 1024
            const uint32_t vslots = smem_u32(s.slots) + kSlots * kSlotBytes;
            const uint64_t pdesc = tc::smem_desc(smem_u32(s.p), 1024, tc::kLayoutSw128);
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t g = 0; ok; ++g) {
                const Tile *d = desc_of(g);
                if (!d) break;
                const int flags = d->flags;
                if (flags & kEnd) break;
                const uint32_t b = g & 1u, vbox = flags & kMixed ? 16 : p.vbox, vsh = 31 - __clz(vbox);
                const uint64_t vdesc = tc::smem_desc_lbo(vslots, vbox * 128, 1024, tc::kLayoutSw128);
                if (!bar_wait(smem_u32(s.pfull + b), (g >> 1) & 1u, p.ctx, s.abort_flag)) break;
#pragma unroll 1
                for (int w = 0; w < Lt::kPieces; ++w, ++it) {
                    const uint32_t sl = it % kSlots;
                    if (!(ok = bar_wait(smem_u32(s.full + kSlots + sl), (it / kSlots) & 1u, p.ctx, s.abort_flag))) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int k = 0; k < Lt::kVKeys / 16; ++k) {  // 16 keys each
                        const uint32_t kt = w * (Lt::kVKeys / 16) + k, x = k * 16;
                        const uint32_t voff = ((((x >> vsh) * Lt::kVChunks) << vsh) + (x & (vbox - 1))) * 128;
#pragma unroll
                        for (int i = 0; i < Lt::kPvMmas; ++i)
                            tc::mma_f16_2sm(tmem + i * (Lt::kPvN / 2),
                                            pdesc + ((b * kPBytes + (kt >> 2) * 8192 + (kt & 3) * 32) >> 4),
                                            vdesc + ((sl * kSlotBytes + voff + i * 2 * vbox * 128) >> 4), p.idesc_pv,
                                            (!(flags & kFirst) || kt) ? 1u : 0u);
                    }
                    tc::mma_commit_2sm(smem_u32(s.empty + kSlots + sl));
                }
                if (!ok) break;
                tc::mma_commit_2sm(smem_u32(s.pvdone + b));
            }
        }
        else if (rank == 1) {
            // -------------------------------------------------------- own rows into L2
            // (by TMA, 16 rows x half the dims each: a prefetch per 128 bytes took longer than the tiles)
            for (uint32_t g = 0;; ++g) {
                const Tile *d = warp_desc_of(g);
                if (!d) break;
                const int flags = d->flags;
                if (!(flags & (kEnd | kShared)) && tc::elect_one())
                    for (int i = 0; i < 8; ++i) {
                        const int row = d->rows[i];
                        if (row < 0) continue;
                        const CUtensorMap *map = (flags >> (kRingShift + i)) & 1 ? &maps.rv16 : &maps.v16;
                        tc::tma_prefetch_3d(map, 0, row, 0);
                        tc::tma_prefetch_3d(map, 0, row, Lt::kVChunks);
                    }
                __syncwarp();
                mbar_arrive(smem_u32(s.dempty + g % kDescs), lane == 0);
                if (flags & kEnd) break;
            }
        }
    } else if (warp == kQueryWarp) {
        // ------------------------------------------------------------ query tiles
        const uint32_t qland = tc::map_to_rank(smem_u32(s.qland), rank), qready0 = tc::map_to_rank(smem_u32(s.qready), 0);
        if (p.dependent) asm volatile("griddepcontrol.wait;" ::: "memory");
        uint32_t nq = 0;
        bool ok = true;
        for (uint32_t g = 0; ok; ++g) {
            const Tile *d = warp_desc_of(g);
            if (!(ok = d != nullptr)) break;
            const int flags = d->flags, row = d->rt() * kPrefixRows + rank * 64;
            __syncwarp();
            mbar_arrive(smem_u32(s.dempty + g % kDescs), lane == 0);
            if (flags & kEnd) break;
            if (!(flags & kFirst)) continue;
            if (!(ok = warp_wait(smem_u32(s.qempty), (nq & 1u) ^ 1u, p.ctx, s.abort_flag))) break;
            if (tc::elect_one()) {
                mbar_arrive_expect_tx_cluster(qland, Lt::kQBytes);
#pragma unroll 1
                for (int c = 0; c < DP / 64; c += 2)
                    tc::tma_load_3d_2sm(smem_u32(s.q) + c * 8192, &maps.q, qland, 0, row, c);
            }
            __syncwarp();
            if (!(ok = warp_wait(smem_u32(s.qland), nq & 1u, p.ctx, s.abort_flag))) break;
            mbar_arrive_cluster(qready0, lane == 0);
            ++nq;
        }
        copies = !ok;
    } else if (warp == kPlanWarp) {
        // ------------------------------------------------------------ planner
        Units un = deal_units(p, reinterpret_cast<const int2 *>(s.p), pair, blockIdx.x == 0);
        uint32_t g = 0;
        bool ok = true;
        // An entry is free for tile g once tile g - kDescs is done with everywhere: once the
        // softmax warps are done with tile g - kDescs + 2, whose P went where the P of that tile was.
        // With one V slot a tile (DP = 128) a V producer passes every other tile by, and the phase of an
        // entry's barrier must not get two ahead of it (it would wait for good): one tile more, so that
        // P.V of the tile after, which that producer brought, is over.
        constexpr uint32_t kDone = Lt::kPieces == 1 ? 3 : 2;
        const auto entry = [&]() -> Tile * {
            const uint32_t t = g + kDone;
            if (t >= kDescs) ok = warp_wait(smem_u32(s.dempty + t % kDescs), (t / kDescs + 1) & 1u, p.ctx, s.abort_flag);
            return ok ? s.desc + g % kDescs : nullptr;
        };
        const auto publish = [&] {
            __syncwarp();
            mbar_arrive(smem_u32(s.dfull + g % kDescs), lane == 0);
            ++g;
        };
        const int win_rows = (int)a.win_rows;
        bool counted = true;  // un.n are the row tile's
        while (un.left > 0 && ok && un.rt < p.plan.row_tiles) {
            const Queries qs = queries_of(p, un.rt);
            const int b0 = p.nq.div(qs.bq0), b1 = p.nq.div(qs.bq1);
            const auto query0 = [&](int b) { return std::max(qs.bq0, b * a.nq); };
            const auto query1 = [&](int b) { return std::min(qs.bq1, b * a.nq + a.nq - 1); };
            // own keys of request bw + lane, 32 requests at a time
            Own mine = {0, 0u};
            int bw = b0 - 32;
            const auto window = [&](int b) {
                bw = b;
                mine = b + lane <= b1 ? own_keys(p, query0(b + lane), query1(b + lane)) : Own{0, 0u};
            };
            if (!counted) {
                int vmax = 0, tiles = 0;
#pragma unroll 1
                for (int q = qs.bq0 + lane; q <= qs.bq1; q += 32) vmax = std::max(vmax, visible(p, __ldg(a.q_pos + q), p.n_shared));
#pragma unroll 1
                for (int b = b0; b <= b1; b += 32) {
                    window(b);
                    tiles += mine.tiles();
                }
                if (bw != b0) window(b0);
                un.n.y = __reduce_max_sync(0xffffffffu, vmax);
                un.n.x = (int)__reduce_add_sync(0xffffffffu, tiles) + (un.n.y + kPrefixKeys - 1) / kPrefixKeys;
            }
            counted = false;
            const int vmax = un.n.y, shared = (vmax + kPrefixKeys - 1) / kPrefixKeys;
            const int n = std::min(un.n.x - un.x, un.left);
            un.left -= std::max(n, 0);
            int x = un.x, b = b0 - 1;
            int y = x - shared;  // the tile's number among its request's own ones
            Own own = {0, 0u};
            for (int j = 0; j < n; ++j, ++x, ++y) {
                const bool sh = x < shared;
                int flags = (sh ? kShared : 0) | (j == 0 ? kFirst : 0) | (j == n - 1 ? kLast : 0);
                int ent, e_first, r_first = 0;
                const int *table = a.table;
                if (sh) {
                    e_first = x * kPrefixKeys;
                    ent = std::min(vmax - e_first, +kPrefixKeys);
                } else {
                    while (y >= own.tiles() && b <= b1) {
                        y -= own.tiles();
                        if (++b >= bw + 32) window(b);
                        own = {__shfl_sync(0xffffffffu, mine.n_own, b - bw), __shfl_sync(0xffffffffu, mine.total, b - bw)};
                    }
                    const int first = y * kPrefixKeys;
                    e_first = p.n_shared + first;
                    ent = std::min(std::max(own.n_own - first, 0), +kPrefixKeys);
                    r_first = first - (int)own.ring0();
                    if (r_first > -kPrefixKeys) flags |= kMixed;
                    table += (size_t)b * a.max_pages;
                }
                // 16 keys by lane: their first row (its page's load flies while an entry is awaited)
                const int k16 = lane * 16, e16 = e_first + k16;
                int id = 0, off = 0;
                if (lane < 8 && k16 < ent) {
                    const int pg = p.page.div(e16);
                    off = e16 - pg * a.page;
                    id = __ldg(table + pg);
                }
                Tile *d = entry();
                if (!d) break;
                int row = -kPrefixKeys;
                bool missing = false, from_ring = false;
                if (lane < 8) {
                    const int rr = r_first + k16;
                    if (k16 < ent) {
                        missing = id < 0 || id >= a.n_pages;
                        if (sh && p.linear) row = e16;
                        else if (p.linear) row = p.n_shared + b * p.own_cap + (e16 - p.n_shared);
                        else if (!missing) row = id * a.page + off;
                    } else if ((flags & kMixed) && rr >= 0 && rr < win_rows) {
                        row = b * win_rows + rr + (p.linear ? p.n_shared + p.batch * p.own_cap : 0);
                        from_ring = true;
                    }
                    d->rows[lane] = row;
                }
                const uint32_t miss = __ballot_sync(0xffffffffu, missing), rings = __ballot_sync(0xffffffffu, from_ring);
                flags |= (int)(miss << kMissingShift) | (int)(rings << kRingShift);
                if (lane < 4) {
                    // 32 keys by lane: which ones a copy brings that no row takes.  Of entries the
                    // last box's rest; of window rows those in no query's window and past the ring.
                    const int vb = flags & kMixed ? 16 : p.vbox, k32 = lane * 32;
                    uint32_t z;
                    z = bits_between(ent - k32, ((ent + vb - 1) & -vb) - 1 - k32);
                    const uint32_t two = rings >> (2 * lane);
                    const uint32_t wins = (two & 1u ? 0x0000ffffu : 0u) | (two & 2u ? 0xffff0000u : 0u);
                    if (wins) {
                        uint32_t live = 0u;
                        const int q1 = query1(b), k0 = r_first + k32;
#pragma unroll 1
                        for (int q = query0(b); q <= q1; ++q) {
                            const int t = __ldg(a.q_pos + q);
                            if (t >= 0) live |= ring_bits(p, window_of(p, t), k0);
                        }
                        z = (z & ~wins) | (wins & ~live);
                    }
                    d->zero[lane] = z;
                }
                if (lane == 0) {
                    d->flags = flags;
                    d->ent_rt = (int)((uint32_t)ent | (uint32_t)un.rt << 8);
                    d->n = n;
                    d->b = b;
                    d->e_first = e_first;
                    d->r_first = r_first;
                }
                publish();
            }
            ++un.rt;
            un.x = 0;
        }
        if (ok) {
            Tile *d = entry();
            if (d) {
                if (lane == 0) d->flags = kEnd;
                publish();
            }
        }
        tc::cluster_wait();
    } else {
        // ------------------------------------------------------------ softmax, partial rows
        // Group wg takes the tiles of its parity; both meet where a row tile begins and ends.
        const int quarter = warp & 3, wg = (warp - kSoftWarp0) >> 2;
        const int tl = quarter * 32 + lane;     // tensor-memory lane
        const int r = tl & 63, hf = tl >> 6;    // row of this CTA's 64; first / second half of the columns
        const int q4 = hf * 2 + wg;             // which of the row's four threads
        volatile uint32_t *xch = s.xch + (quarter & 1) * 128;                     // of these 32 rows
        float *sums = reinterpret_cast<float *>(s.p + (quarter & 1) * 4096);      // [4][32], where none of their P is
        const uint32_t rbar = smem_u32(s.rbar + (quarter & 1));
        uint32_t rbar_n = 0;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t sempty0 = tc::map_to_rank(smem_u32(s.sempty), 0), pfull0 = tc::map_to_rank(smem_u32(s.pfull), 0);
        const int n_rows = (int)(a.n_bq * a.H);
        if (p.dependent) asm volatile("griddepcontrol.wait;" ::: "memory");
        uint32_t nq = 0;
        Row rw = {-1, 0, 0, {0, 0}};
        int vis_min = 0;  // the fewest entries that a row of this warp sees
        // The rows' reference m follows the maxima of all tiles, of either group; l is relative to m_l.
        float rq = 0.f, m = -INFINITY, m_l = -INFINITY, l = 0.f;
        // The row's maximum in tile g, once both halves of it are there.  A poll of the words
        // themselves: an mbarrier between the two warps took ~400 cycles.
        const auto tile_max = [&](uint32_t g, float &mt) {
            const uint32_t at = (g & 1u) * 64 + lane, tag = tag_of(g);
            uint64_t t0 = 0;
            for (int i = 0;; ++i) {
                const uint32_t x = xch[at], y = xch[at + 32];
                if (__all_sync(0xffffffffu, (x & kTagMask) == tag && (y & kTagMask) == tag)) {
                    mt = fmaxf(untagged(x), untagged(y));
                    return true;
                }
                if ((i & 63) == 63) {
                    const uint64_t now = global_timer_ns();
                    if (t0 == 0) t0 = now;
                    if (now - t0 > p.ctx.budget_ns) {
                        record_status(p.ctx.status, CSA_ERR_TIMEOUT);
                        *(volatile int *)s.abort_flag = 1;
                    }
                    if (__any_sync(0xffffffffu, *(volatile int *)s.abort_flag)) return false;
                }
            }
        };
        const auto raise = [](float m0, float mt) { return m0 == -INFINITY || mt > m0 + kRescaleThreshold ? mt : m0; };
        const auto wait = [&](uint64_t *bar, uint32_t parity) {
            return warp_wait(smem_u32(bar), parity, p.ctx, s.abort_flag);
        };
        for (uint32_t g0 = 0;;) {
            const Tile *d0 = warp_desc_of(g0);  // the first tile of a part
            if (!d0 || (d0->flags & kEnd)) break;
            const uint32_t last = g0 + (uint32_t)d0->n - 1u;
            const size_t part = (size_t)pair + d0->rt();
            const int row = d0->rt() * kPrefixRows + rank * 64 + r;
            const int bq = row < n_rows ? p.H.div(row) : 0;
            rw.t = row < n_rows ? __ldg(a.q_pos + bq) : -1;
            rw.b = p.nq.div(bq);
            rw.vis = visible(p, rw.t, (int)a.N);
            rw.w = window_of(p, std::max(rw.t, 0));
            vis_min = __reduce_min_sync(0xffffffffu, rw.vis);
            if (!wait(s.qland, nq & 1u)) break;
            ++nq;
            if (!p.lo) sums[q4 * 32 + lane] = query_squares<DP>(s.q, r, q4);
            __syncwarp();
            mbar_arrive(smem_u32(s.qempty), lane == 0);
            if (!warps_meet(rbar, rbar_n, p.ctx, s.abort_flag)) break;
            if (p.lo) {
                if (row < n_rows) rq = p.rq[row];
            } else {
                const float ss = (sums[lane] + sums[32 + lane]) + (sums[64 + lane] + sums[96 + lane]);
                rq = row_factor(a, ss);
            }
            if (rw.t < 0) rq = 1.f;  // an empty slot's query may hold anything: no NaN for its masked scores
            m = m_l = -INFINITY;
            l = 0.f;
            if (!warps_meet(rbar, rbar_n, p.ctx, s.abort_flag)) break;
            // this group's tiles
            bool ok = true;
            for (uint32_t g = g0 + ((g0 ^ (uint32_t)wg) & 1u); g <= last; g += 2) {
                ok = false;  // until the tile is done
                const Tile *dp = warp_desc_of(g);
                if (!dp) break;
                const Tile &d = *dp;
                const int flags = d.flags;
                const uint32_t b = g & 1u, ph = (g >> 1) & 1u, sb = g % kSBufs;
                uint32_t mk0 = 0xffffffffu, mk1 = 0xffffffffu;  // keys that take part
                bool whole = (flags & (kShared | 0xff << kMissingShift)) == kShared && d.ent() == kPrefixKeys &&
                             d.e_first + kPrefixKeys <= vis_min;
                if (!whole) {
                    mk0 = key_mask(p, d, hf * 64, rw);
                    mk1 = key_mask(p, d, hf * 64 + 32, rw);
                    whole = __all_sync(0xffffffffu, (mk0 & mk1) == 0xffffffffu);
                }
                if ((mk0 | mk1) && l == 0.f) l = kTaken;
                if (!wait(s.sfull + sb, (g / kSBufs) & 1u)) break;
                tc::fence_after_sync();
                float sc[64];
                tc::tmem_ld32(tmem + lane_base + kSCols + sb * 64, sc);
                tc::tmem_ld32(tmem + lane_base + kSCols + sb * 64 + 32, sc + 32);
                tc::tmem_wait_ld();
                tc::fence_before_sync();
                __syncwarp();
                mbar_arrive_cluster(sempty0 + sb * 8, lane == 0);
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) sc[i] = ((i < 32 ? mk0 : mk1) >> (i & 31)) & 1u ? sc[i] : -INFINITY;
                }
                float m2[2] = {sc[0], sc[1]};
#pragma unroll
                for (int i = 2; i < 64; i += 2) {
                    m2[0] = fmaxf(m2[0], sc[i]);
                    m2[1] = fmaxf(m2[1], sc[i + 1]);
                }
                float mt = fmaxf(m2[0], m2[1]) * rq;
                // The row's maximum over its two threads (any reference near the maximum serves, as long
                // as all four agree).  A word is written again two tiles on: by then this tile's P.V is
                // over, for which the partner has read it, and the other group has written the tile's
                // between, before which it has.
                if (!wait(s.pvdone + b, ph ^ 1u)) break;  // (P buffer b is free, too)
                float other;
                if (g > g0) {
                    if (!tile_max(g - 1, other)) break;
                    m = raise(m, other);
                } else if (g > 0 && !tile_max(g - 1, other)) {
                    break;
                }
                xch[b * 64 + hf * 32 + lane] = tagged(mt, g);
                if (!tile_max(g, mt)) break;
                const float m_old = m;
                const bool mine = m != -INFINITY && mt > m + kRescaleThreshold;
                m = raise(m, mt);
                if (__any_sync(0xffffffffu, mine)) {
                    const uint32_t gp = g - 1;  // O after the P.V of the tile before
                    if (!wait(s.pvdone + (gp & 1u), (gp >> 1) & 1u)) break;
                    tc::fence_after_sync();
                    const float f = mine ? exp2f(m_old - m) : 1.0f;
#pragma unroll 1
                    for (int c = 0; c < DP / 2; c += 16) {
                        float v[16];
                        tc::tmem_ld16(tmem + lane_base + c, v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] *= f;
                        tc::tmem_st16(tmem + lane_base + c, v);
                    }
                    tc::tmem_wait_st();
                }
                if (m_l != m) {
                    if (m_l != -INFINITY) l *= exp2f(m_l - m);
                    m_l = m;
                }
                float mref = m == -INFINITY ? 0.f : m;
                const float sized = difference_scale(mref), factor = rq * sized;
                mref *= sized;
                uint8_t *prow = s.p + b * kPBytes + hf * 8192 + r * 128;
                float ps[2] = {0.f, 0.f};
#pragma unroll
                for (int x = 0; x < 8; ++x) {  // 8 keys: 16 bytes
                    float e[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) e[i] = exp2_ftz(fmaf(sc[x * 8 + i], factor, -mref));
                    // l sums the weights as they are rounded: what the rounding changes in common cancels
                    // in O / l (of a row with one key, all of it)
                    const uint4 w = pack8(e);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ps[0] += __uint_as_float(ww[i] << 16);
                        ps[1] += __uint_as_float(ww[i] & 0xffff0000u);
                    }
                    *reinterpret_cast<uint4 *>(prow + ((x ^ (r & 7)) << 4)) = w;
                }
                l += ps[0] + ps[1];
                tc::fence_proxy_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                mbar_arrive_cluster(pfull0 + b * 8, lane == 0);
                __syncwarp();
                mbar_arrive(smem_u32(s.dempty + g % kDescs), lane == 0);
                ok = true;
            }
            if (!ok) break;
            const uint32_t lb = last & 1u, lph = (last >> 1) & 1u;
            if (lb != (uint32_t)wg) {
                // The last tile's maxima, too.  They were written after the P.V before it of its parity was
                // over, so that lph is the phase awaited below (waiting for that one here would be a wait for
                // good once the last P.V is over, too).
                float other;
                if (!tile_max(last, other)) break;
                m = raise(m, other);
            }
            if (!wait(s.pvdone + lb, lph)) break;
            tc::fence_after_sync();
            if (m_l != m && m_l != -INFINITY) l *= exp2f(m_l - m);
            if (!warps_meet(rbar, rbar_n, p.ctx, s.abort_flag)) break;
            sums[q4 * 32 + lane] = l;
            if (!warps_meet(rbar, rbar_n, p.ctx, s.abort_flag)) break;
            if (q4 == 0)
                p.ml[part * kPrefixRows + rank * 64 + r] =
                    partial_ml(m, (sums[lane] + sums[32 + lane]) + (sums[64 + lane] + sums[96 + lane]));
            if (!warps_meet(rbar, rbar_n, p.ctx, s.abort_flag)) break;
            float4 *dst = reinterpret_cast<float4 *>(p.part) + (part * 2 + rank) * (DP / 8) * 128 + tl;
#pragma unroll 1
            for (int c = wg * (DP / 4); c < (wg + 1) * (DP / 4); c += 32) {
                float v[32];
                tc::tmem_ld32(tmem + lane_base + c, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dst[(size_t)(c / 4 + i) * 128] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
            tc::fence_before_sync();  // O is read before the next row tile's first P.V (through pfull)
            g0 = last + 1u;
        }
    }
    if (copies) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();  // no arrival of the other CTA is outstanding
    if (warp == kQueryWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc_2sm(tmem, 512);
    }
}

// 8 floats of a table that may be aligned to 4 bytes only (`wide`: to 16)
CSA_DEVINL void load8(const float *p, bool wide, float x[8]) {
    if (wide) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __ldg(p + e);
    }
}

// Query rows under a gain, the scale's sign and RoPE (channel D-64+j of the slice
// rotates with D-32+j), as hi + lo in bf16, and their factors.  A warp per row.
__global__ void __launch_bounds__(256)
    query_rows_kernel(const AttendArgs a, const FastDiv H, int n_rows, uint16_t *__restrict__ hi, uint16_t *__restrict__ lo,
                      float *__restrict__ rq) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, row = (int)(blockIdx.x * 8 + (threadIdx.x >> 5)), units = a.D / 8;
    if (row >= n_rows) return;
    const float sign = a.scale < 0.f ? -1.f : 1.f;
    const long long t = __ldg(a.q_pos + H.div(row));
    // (4-byte loads of the gain, 16 a lane and row, took more of L1 than the rows themselves)
    const bool wide = ((reinterpret_cast<uintptr_t>(a.q_gain) | reinterpret_cast<uintptr_t>(a.rope_cos) |
                        reinterpret_cast<uintptr_t>(a.rope_sin)) & 15u) == 0;
    const bool turns = a.rope_cos && t >= 0 && t < a.rope_npos;
    const uint4 *src = reinterpret_cast<const uint4 *>(a.q) + (size_t)row * units;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // units lane, lane + 32 (D = 512); the rotated ones are the last 8 of a row
        const int u = lane + i * 32;
        if (i * 32 >= units) break;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (u < units) unpack8(ldg16(src + u), x);
        float gain[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        if (a.q_gain && u < units) load8(a.q_gain + u * 8, wide, gain);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ss = fmaf(x[e], x[e], ss);
            x[e] *= sign * gain[e];
        }
        if (turns) {  // (of the whole warp's row)
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __shfl_xor_sync(0xffffffffu, x[e], 4);
            if (u >= units - 8 && u < units) {
                const bool first = u < units - 4;
                const size_t at = (size_t)t * (kRopeDim / 2) + ((u - (units - 8)) & 3) * 8;
                float c[8], s[8];
                load8(a.rope_cos + at, wide, c);
                load8(a.rope_sin + at, wide, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = first ? x[e] * c[e] - y[e] * s[e] : x[e] * c[e] + y[e] * s[e];
            }
        }
        if (u < units) {
            const uint4 h = pack8(x);
            float back[8];
            unpack8(h, back);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] -= back[e];
            reinterpret_cast<uint4 *>(hi)[(size_t)row * units + u] = h;
            reinterpret_cast<uint4 *>(lo)[(size_t)row * units + u] = pack8(x);
        }
    }
    ss = warp_sum(ss);
    if (lane == 0) rq[row] = row_factor(a, ss);  // (an infinite element is Inf + NaN here: its scores are NaN)
}

// The rows of an FP8 cache that a call reads, as bf16 (exact) in the order of
// PrefixArgs; entries without a page are zero, those that no query sees stay as
// they are (nothing reads them).
struct ExpandParams {
    AttendArgs a;
    int units;  // of 16 codes
    int n_shared, own_cap, batch;
    FastDiv upr, own, page;
    uint4 *out;
};

__global__ void __launch_bounds__(256) expand_rows_kernel(const ExpandParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const AttendArgs &a = p.a;
    const int u = (int)(blockIdx.x * 256 + threadIdx.x);
    if (u >= p.units) return;
    const int row = p.upr.div(u), c = u - row * (int)p.upr.d;
    const int own0 = p.n_shared, ring0 = own0 + p.batch * p.own_cap;
    const uint8_t *codes = a.kv8, *exps = a.kv8e;
    long long src = -1;
    if (row >= ring0) {
        src = row - ring0;
        codes = a.win8;
        exps = a.win8e;
    } else {
        int e = row, b = 0;
        if (row >= own0) {
            b = p.own.div(row - own0);
            e = own0 + (row - own0) - b * p.own_cap;
            int t = -1;
            for (int i = 0; i < a.nq; ++i) t = max(t, __ldg(a.q_pos + (size_t)b * a.nq + i));
            if (e >= n_visible(t, a.m, a.N)) return;
        }
        const int pg = p.page.div(e), id = __ldg(a.table + (size_t)b * a.max_pages + pg);
        if (id >= 0 && id < a.n_pages) src = (long long)id * a.page + (e - pg * a.page);
    }
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (src >= 0) {
        const uint4 v = ldg_stream(codes + src * a.D + c * 16);
        const uint32_t e = __ldg(exps + src * (a.D / 128) + c / 8);
        lo = e4m3x8_bf16x8(make_uint2(v.x, v.y), e);
        hi = e4m3x8_bf16x8(make_uint2(v.z, v.w), e);
    }
    p.out[2 * (size_t)u] = lo;
    p.out[2 * (size_t)u + 1] = hi;
}

// kind::f16 instruction descriptor: bf16 operands, fp32 accumulate, M = 128
constexpr uint32_t idesc(int n, bool b_mn) { return tc::idesc_f16(n, true) | (b_mn ? (1u << 16) : 0u); }

template <int DP>
int launch_d(const PrefixArgs &x, const DevCtx &ctx, cudaStream_t st) {
    Params p = {};
    p.a = x.a;
    p.plan = x.plan;
    p.n_shared = (int)x.n_shared;
    p.linear = x.own_cap >= 0 ? 1 : 0;
    p.lo = x.lo ? 1 : 0;
    p.rq = x.rq;
    p.dependent = p.linear || p.lo;
    p.batch = (int)(x.a.n_bq / x.a.nq);
    p.own_cap = x.own_cap;
    p.part = x.part;
    p.ml = x.ml;
    p.meet = x.meet;
    p.H = FastDiv::by((uint32_t)x.a.H);
    p.nq = FastDiv::by((uint32_t)x.a.nq);
    p.m = FastDiv::by((uint32_t)x.a.m);
    p.page = FastDiv::by((uint32_t)x.a.page);
    p.ring = FastDiv::by((uint32_t)x.a.win_rows);
    p.ctx = ctx;
    p.idesc_qk = idesc(kPrefixKeys, false);
    p.idesc_pv = idesc(Layout<DP>::kPvN, true);
    p.box = p.linear || x.a.page % 64 == 0 ? 64 : (x.a.page % 32 == 0 ? 32 : 16);
    p.vbox = std::min(p.box, Layout<DP>::kVKeys);
    auto kern = attend_prefix_kernel<DP>;
    constexpr size_t smem = smem_bytes<DP>();
    static SmemSet smem_set;
    if (!smem_set((const void *)kern, smem)) return CSA_ERR_CUDA;
    // [64-dim chunk][row][64]: one copy brings several chunks of its rows (past D: zeros)
    const auto encode = [&](CUtensorMap *map, const uint16_t *base, long long rows, int box_rows, int chunks) {
        const uint64_t dims[3] = {64, (uint64_t)rows, (uint64_t)(x.a.D / 64)};
        const uint64_t strides[2] = {(uint64_t)x.a.D * 2, 128};
        const uint32_t box[3] = {64, (uint32_t)box_rows, (uint32_t)chunks};
        return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                                 CU_TENSOR_MAP_SWIZZLE_128B);
    };
    const long long batch = p.batch, rings = batch * x.a.win_rows;
    const long long key_rows = p.linear ? x.n_shared + batch * x.own_cap + rings : x.a.n_pages * x.a.page;
    constexpr int kChunks = Layout<DP>::kVChunks;
    Maps maps = {};
    if (!encode(&maps.q, x.lo ? x.hi : x.a.q, x.a.n_bq * x.a.H, 64, 2) ||
        (x.lo && !encode(&maps.lo, x.lo, x.a.n_bq * x.a.H, 64, 2)) ||
        !encode(&maps.k, x.keys, key_rows, p.box, p.box == 64 ? 2 : 1) ||
        !encode(&maps.v, x.keys, key_rows, p.vbox, kChunks))
        return CSA_ERR_CUDA;
    if (!encode(&maps.k16, x.keys, key_rows, 16, 1) || !encode(&maps.v16, x.keys, key_rows, 16, kChunks)) return CSA_ERR_CUDA;
    maps.rk16 = maps.k16;  // (linear: the rings' rows are in the copy, too)
    maps.rv16 = maps.v16;
    if (!p.linear && (!encode(&maps.rk16, x.a.win, rings, 16, 1) || !encode(&maps.rv16, x.a.win, rings, 16, kChunks)))
        return CSA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * x.plan.pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = p.dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, maps, p) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // namespace

PrefixPlan prefix_plan(long long rows) {
    PrefixPlan pl;
    pl.row_tiles = (int)((rows + kPrefixRows - 1) / kPrefixRows);
    pl.pairs = std::max(num_sms() / 2, 1);
    return pl;
}

int launch_query_rows(const PrefixArgs &x, cudaStream_t st) {
    const int rows = (int)(x.a.n_bq * x.a.H);
    query_rows_kernel<<<(unsigned)(rows + 7) / 8, 256, 0, st>>>(x.a, FastDiv::by((uint32_t)x.a.H), rows, x.hi, x.lo, x.rq);
    return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

int launch_expand_rows(const PrefixArgs &x, uint16_t *out, cudaStream_t st) {
    ExpandParams p = {};
    p.a = x.a;
    p.n_shared = (int)x.n_shared;
    p.own_cap = x.own_cap;
    p.batch = (int)(x.a.n_bq / x.a.nq);
    p.upr = FastDiv::by((uint32_t)(x.a.D / 16));
    p.own = FastDiv::by((uint32_t)std::max(x.own_cap, 1));
    p.page = FastDiv::by((uint32_t)x.a.page);
    p.units = (int)((x.n_shared + p.batch * (x.own_cap + x.a.win_rows)) * (x.a.D / 16));  // below 2^25: a limited copy
    p.out = reinterpret_cast<uint4 *>(out);
    expand_rows_kernel<<<(unsigned)(p.units + 255) / 256, 256, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

int launch_attend_prefix(const PrefixArgs &p, const DevCtx &ctx, cudaStream_t st) {
    switch (prefix_dims(p.a.D)) {
        case 128: return launch_d<128>(p, ctx, st);
        case 256: return launch_d<256>(p, ctx, st);
        case 512: return launch_d<512>(p, ctx, st);
        default: return CSA_ERR_UNSUPPORTED;
    }
}

}  // namespace csa
