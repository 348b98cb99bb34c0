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
// heads shares the tile's tensor work that the mask throws away.  O, m and l of
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
// The tensor cores' operand reads (224 KiB), these loads and P share the
// 128 B/cycle of shared memory, which bounds the kernel at D = 512.
//
// Warps: 0 and 1 producers of K, 2 and 3 of V, 4 and 5 MMA issuers of Q K^T and of
// P V on the pair's leader (one thread for both was busy for longer than the
// tensor cores: a satisfied barrier wait takes ~140 cycles, an MMA ~20), 6
// tensor memory and the query tiles, 7 the planner, 8..15 softmax (four threads
// per row: lane half x 32-column half).
// The planner walks the pair's tiles a few ahead of everyone, describes each in
// shared memory (struct Tile) and brings own rows into L2 (the producers are one
// tile ahead at D = 512).  Each role's code is kept small on purpose: unrolled
// loops that run once per row tile cost more in instruction misses than in work
// (14K cycles per row tile, measured, for a prologue of ~3K instructions).
// K and V have a ring of 16 KiB slots each; every tile passes through both, and
// two producer warps take a ring's positions in turn, whatever they hold: shared
// entries by TMA, own keys (rows of any page and of the window rings) by 16-byte
// asynchronous copies, FP8 rows expanded on the way.  (A slot's phase bit tells
// its use from the one before only: whoever waits on a ring passes every use.)
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
constexpr int kDescs = 8;  // tiles described ahead
constexpr uint32_t kSlotBytes = 16384;  // K: 64 keys x 128 dims, V: 16384 / DP keys x DP / 2 dims
constexpr uint32_t kPBytes = 16384;     // 64 rows x 128 keys, bf16
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t kSCols = 256;        // first column of the S buffers (64 columns each)

template <int DP>
struct Layout {
    static constexpr int kPieces = DP / 128;              // slots of a K tile, and of a V tile, per SM
    static constexpr int kPvN = DP < 256 ? DP : 256;      // N of one P.V MMA
    static constexpr int kPvMmas = DP / kPvN;             // MMAs per 16 keys
    static constexpr int kVKeys = 16384 / DP;             // keys of a V slot
    static constexpr int kVChunks = DP / 128;             // its 64-dim chunks (this SM's half of V's columns)
    static constexpr uint32_t kQBytes = 64 * DP * 2;      // [DP/64][64 rows][128 B]
};

struct Params {
    AttendArgs a;
    PrefixPlan plan;
    int n_shared;
    int linear;
    long long *first; // [row_tiles + 1] first unit of a row tile; the units of all
    int box;          // entries that one copy brings at most (none crosses a page): 16, 32 or 64
    int vbox;         // those of a V copy: at most one slot's
    float *part;
    float2 *ml;
    uint32_t idesc_qk, idesc_pv;
    DevCtx ctx;
};

// One tile of 128 keys, as the planner describes it.
enum : int { kShared = 1, kFirst = 2, kLast = 4, kEnd = 8, kMissingShift = 8 };
struct __align__(16) Tile {
    int flags;    // kShared: entries of all requests, else own keys; kFirst / kLast of a pair's part of a
                  // row tile; kEnd: no tile.  Bit kMissingShift + i: entries 16 i .. 16 i + 15 have no page
    int rt;       // row tile
    int b;        // request (own keys)
    int e_first;  // entry index of key 0 (own keys: may pass the last entry)
    int ent;      // keys [0, ent) are entries that some row sees
    int cnt;      // keys [ent, cnt) are window rows, of position
    int wpos;     //   wpos + key
    int ring;     // their row in the request's ring: (ring + key - ent) % win_rows
    int rows[8];  // pool row (linear: row of the copy) of entry 16 i; < 0: none, reads as zeros
};

struct Smem {
    uint8_t *q, *slots, *p;  // slots: K's ring, then V's; so are their barriers
    uint64_t *full, *empty, *sfull, *sempty, *pfull, *pvdone, *qland, *qready, *qempty, *vfix, *dfull, *dempty;
    Tile *desc;      // [kDescs]
    uint16_t *xmax;  // [2][4][64] the upper halves of the row maxima of a tile's four threads per row
    float *xsum;     // [4][64], the same memory
    uint32_t *tmem_slot;
    int *abort_flag;
};

template <int DP>
CSA_DEVINL Smem carve(uint8_t *raw) {
    Smem s;
    s.q = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    s.slots = s.q + Layout<DP>::kQBytes;
    s.p = s.slots + 2 * kSlots * kSlotBytes;
    s.xsum = reinterpret_cast<float *>(s.p + 2 * kPBytes);
    s.xmax = reinterpret_cast<uint16_t *>(s.xsum);
    s.desc = reinterpret_cast<Tile *>(s.xsum + 256);
    uint64_t *bars = reinterpret_cast<uint64_t *>(s.desc + kDescs);
    s.full = bars;
    s.empty = s.full + 2 * kSlots;
    s.dfull = s.empty + 2 * kSlots;
    s.dempty = s.dfull + kDescs;
    s.sfull = s.dempty + kDescs;
    s.sempty = s.sfull + 2;
    s.pfull = s.sempty + 2;
    s.pvdone = s.pfull + 2;
    s.qland = s.pvdone + 2;
    s.qready = s.qland + 1;
    s.qempty = s.qready + 1;
    s.vfix = s.qempty + 1;  // [2]
    s.tmem_slot = reinterpret_cast<uint32_t *>(s.vfix + 2);
    s.abort_flag = reinterpret_cast<int *>(s.tmem_slot + 1);
    return s;
}

template <int DP>
constexpr size_t smem_bytes() {
    return 1024 + Layout<DP>::kQBytes + 2 * kSlots * kSlotBytes + 2 * kPBytes + 1024 + kDescs * sizeof(Tile) +
           (4 * kSlots + 2 * kDescs + 13) * 8 + 8;
}
static_assert(smem_bytes<512>() <= 227 * 1024, "shared memory of one CTA");

// ---------------------------------------------------------------- units
// The tiles of row tile rt, in order: the shared entries that any of its rows
// sees, then request by request the own keys of its queries in the row tile.
CSA_DEVINL int visible(const Params &p, int t, int cap) {
    const uint32_t v = t < 0 ? 0u : ((uint32_t)t + 1u) / (uint32_t)p.a.m;
    return v < (uint32_t)cap ? (int)v : cap;
}

// The own keys of queries [q0, q1] of one request: entries n_shared..n_shared + n_own - 1,
// then the window rows of positions u0..u0 + (total - n_own) - 1.
struct Own {
    int n_own, u0;
    long long total;
    CSA_DEVINL int tiles() const { return (int)((total + kPrefixKeys - 1) / kPrefixKeys); }
};

CSA_DEVINL Own own_keys(const Params &p, int q0, int q1) {
    int vis = 0, u0 = 0x7fffffff, u1 = -1;
    for (int q = q0; q <= q1; ++q) {
        const int t = __ldg(p.a.q_pos + q);
        if (t < 0) continue;
        vis = std::max(vis, visible(p, t, (int)p.a.N));
        u0 = std::min(u0, std::max(0, t - p.a.W + 1));
        u1 = std::max(u1, t);
    }
    Own o;
    o.n_own = std::max(0, vis - p.n_shared);
    o.u0 = u0;
    o.total = o.n_own + (u1 >= 0 ? (long long)u1 - u0 + 1 : 0);
    return o;
}

// Queries (rows of q_pos) bq0..bq1 of row tile rt.
struct Queries {
    int bq0, bq1;
};

CSA_DEVINL Queries queries_of(const Params &p, int rt) {
    Queries r;
    const uint32_t row0 = (uint32_t)rt * kPrefixRows, H = (uint32_t)p.a.H;
    r.bq0 = (int)(row0 / H);
    r.bq1 = (int)std::min<uint32_t>((uint32_t)p.a.n_bq - 1, (row0 + kPrefixRows - 1) / H);
    return r;
}

// Units of row tile rt, by `subs` consecutive lanes that share its requests (the
// sum is every lane's); rt past the last: 0.
CSA_DEVINL int count_units(const Params &p, int rt, int subs) {
    int vmax = 0, n = 0;
    if (rt < p.plan.row_tiles) {
        const Queries r = queries_of(p, rt);
        const int b1 = r.bq1 / p.a.nq;
        for (int b = r.bq0 / p.a.nq + (threadIdx.x & (subs - 1)); b <= b1; b += subs) {
            const int q0 = std::max(r.bq0, b * p.a.nq), q1 = std::min(r.bq1, b * p.a.nq + p.a.nq - 1);
            n += own_keys(p, q0, q1).tiles();
            for (int q = q0; q <= q1; ++q) vmax = std::max(vmax, visible(p, __ldg(p.a.q_pos + q), p.n_shared));
        }
    }
    for (int d = 1; d < subs; d <<= 1) {
        n += __shfl_xor_sync(0xffffffffu, n, d);
        vmax = std::max(vmax, __shfl_xor_sync(0xffffffffu, vmax, d));
    }
    return n + (vmax + kPrefixKeys - 1) / kPrefixKeys;
}

// A pair's units: `left` of them from number x of row tile rt on.
struct Units {
    long long left;
    int rt, x;
};

// By one warp; `write`: also where every row tile begins.
CSA_DEVINL Units deal_units(const Params &p, int pair, bool write) {
    const int lane = threadIdx.x & 31, RT = p.plan.row_tiles;
    // lanes per row tile: about its requests
    int subs = 1;
    while (subs < 32 && subs * p.a.H * p.a.nq < kPrefixRows) subs *= 2;
    const int step = 32 / subs;  // row tiles per pass
    long long total = 0;
    int n = 0, inc = 0;
    const auto pass = [&](int r0) {  // n: units of row tile r0 + lane / subs; inc: of those up to it in this pass
        n = count_units(p, r0 + lane / subs, subs);
        inc = n;
        for (int d = subs; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += up;
        }
    };
    for (int r0 = 0; r0 < RT; r0 += step) {
        pass(r0);
        const int rt = r0 + lane / subs;
        if (write && rt < RT && (lane & (subs - 1)) == 0) p.first[rt] = total + inc - n;
        total += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (write && lane == 0) p.first[RT] = total;
    const int P = p.plan.active(total);
    Units u = {0, 0, 0};
    const long long u0 = pair < P ? total * pair / P : 0;
    u.left = pair < P ? total * (pair + 1) / P - u0 : 0;
    if (u.left == 0) return u;
    long long base = 0;
    for (int r0 = 0; r0 < RT; r0 += step) {
        if (RT > step) pass(r0);
        const uint32_t here = __ballot_sync(0xffffffffu, base + inc - n <= u0 && u0 < base + inc);
        if (here) {
            const int l = __ffs(here) - 1;
            u.rt = r0 + l / subs;
            u.x = (int)(u0 - base) - __shfl_sync(0xffffffffu, inc - n, l);
            break;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    return u;
}

CSA_DEVINL bool warp_wait(uint32_t bar, uint32_t parity, const DevCtx &ctx, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctx, abort));
}

CSA_DEVINL void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// ... and whether `v` holds for all of the barrier's threads
CSA_DEVINL bool group_all(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\t"
        "bar.red.and.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((int)v)
        : "memory");
    return r != 0;
}

// The tile's query rows as they landed: this thread's quarter of row r (units
// q4, q4 + 4, .. of 8 dims) -> its sum of squares.
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
    return ss[0] + ss[1];
}

// Rewrites the same units: the gain, then the rotation of the trailing kRopeDim
// channels (unit j of the slice pairs with j + 4, also this thread's); rounded
// to bf16, as the tensor cores' operand is.
template <int DP>
CSA_DEVINL void query_rewrite(const AttendArgs &a, uint8_t *q, int r, int q4, int t) {
    const int r0 = a.D / 8 - kRopeDim / 8;  // first rotated unit
#pragma unroll 1
    for (int unit = q4; unit * 8 < a.D; unit += 8) {
        uint4 *p0 = query_unit<DP>(q, r, unit), *p1 = query_unit<DP>(q, r, unit + 4);
        float x[8], y[8];
        unpack8(*p0, x);
        unpack8(*p1, y);
        if (a.q_gain) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] *= __ldg(a.q_gain + unit * 8 + e);
                y[e] *= __ldg(a.q_gain + unit * 8 + 32 + e);
            }
        }
        if (a.rope_cos && unit >= r0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 cs = rope_cs(a, t, (unit - r0) * 8 + e);
                const float x0 = x[e], y0 = y[e];
                x[e] = x0 * cs.x - y0 * cs.y;
                y[e] = y0 * cs.x + x0 * cs.y;
            }
        }
        *p0 = pack8(x);
        *p1 = pack8(y);
    }
}

// the first n of 32 bits
CSA_DEVINL uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u); }

// Which of keys off..off + 31 of a tile the row of a query at t takes (of
// request b_row, seeing vis entries).
CSA_DEVINL uint32_t key_mask(const Tile &d, int off, int t, int W, int vis, int b_row) {
    if (!(d.flags & kShared) && b_row != d.b) return 0u;
    uint32_t mask = low_bits(std::min(vis - d.e_first, d.ent) - off);
    if (d.flags >> kMissingShift) {
        const int miss = d.flags >> (kMissingShift + off / 16);
        mask &= ~((miss & 1 ? 0x0000ffffu : 0u) | (miss & 2 ? 0xffff0000u : 0u));
    }
    if (d.cnt > d.ent && t >= 0) {  // window rows t-W+1..t
        const int lo = std::max(std::max(0, t - W + 1) - d.wpos, d.ent), hi = std::min(t - d.wpos + 1, d.cnt);
        mask |= low_bits(hi - off) & ~low_bits(lo - off);
    }
    return mask;
}

// One slot of an own tile, by one warp: K (V = false): the CTA's 64 keys x dims
// [128 w, 128 w + 128), V: keys [w kVKeys, ..) x the CTA's half of the dims, in
// the layouts that the TMA copies of shared tiles make.  Keys that do not exist
// are zeros (no weight is on them, and nothing is known of their memory).
template <int DP, bool FP8, bool V>
CSA_DEVINL void gather_slot(const Params &p, const Tile &d, int rank, int w, uint32_t dst) {
    using Lt = Layout<DP>;
    const AttendArgs &a = p.a;
    constexpr int kKeys = V ? Lt::kVKeys : 64, kUnits = V ? Lt::kVChunks * 8 : 16;  // 16-byte units (8 dims) of a key
    constexpr int kPer = FP8 ? 2 : 1;                       // units per thread and step (16 codes)
    constexpr int kStep = 32 * kPer / kUnits;               // keys per step of the warp
    const int lane = threadIdx.x & 31, u = lane % (kUnits / kPer) * kPer;
    const int key0 = V ? w * kKeys : rank * 64, dim = (V ? rank * (DP / 2) : w * 128) + u * 8;
    const int vsh = 31 - __clz(p.vbox);
    const long long ring0 = (long long)d.b * a.win_rows;
    const int rows = (int)a.win_rows;
    // row of key k, ~row in the rings, or none
    constexpr long long kNone = 0x7fffffffffffffffLL;
    const auto row_of = [&](int k) -> long long {
        if (k < d.ent) {
            const int r = d.rows[k >> 4];
            return r < 0 ? kNone : (long long)(r + (k & 15));
        }
        if (k >= d.cnt) return kNone;
        int r = d.ring + (k - d.ent);
        if (r >= rows) r = r - rows < rows ? r - rows : r % rows;
        return ~(ring0 + r);
    };
    // shared-memory address of unit x of the slot's key k: V as [k / vbox][64-dim chunk][k % vbox]
    // [128 B], K as [chunk][k][128 B], 128-byte swizzle
    const auto at = [&](int k, int x) {
        const uint32_t line = V ? ((uint32_t)((k >> vsh) * Lt::kVChunks + (x >> 3)) << vsh) + (k & (p.vbox - 1))
                                : (uint32_t)((x >> 3) * 64 + k);
        return dst + line * 128 + (((x & 7) ^ (k & 7)) << 4);
    };
    if constexpr (FP8) {
        constexpr int kBatch = 4;
#pragma unroll 1
        for (int k0 = lane / (kUnits / 2); k0 < kKeys; k0 += kBatch * kStep) {
            uint4 v[kBatch];
            uint32_t e[kBatch];
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
                const long long r = row_of(key0 + k0 + c * kStep);
                v[c] = make_uint4(0u, 0u, 0u, 0u);
                e[c] = 0u;
                if (r != kNone) {
                    const size_t ri = (size_t)(r < 0 ? ~r : r);
                    v[c] = ldg16((r < 0 ? a.win8 : a.kv8) + ri * a.D + dim);
                    e[c] = __ldg((r < 0 ? a.win8e : a.kv8e) + ri * (a.D / 128) + dim / 128);
                }
            }
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
                const int k = k0 + c * kStep;
                const uint4 lo = e4m3x8_bf16x8(make_uint2(v[c].x, v[c].y), e[c]);
                const uint4 hi = e4m3x8_bf16x8(make_uint2(v[c].z, v[c].w), e[c]);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(k, u)), "r"(lo.x), "r"(lo.y), "r"(lo.z),
                             "r"(lo.w)
                             : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(k, u + 1)), "r"(hi.x), "r"(hi.y), "r"(hi.z),
                             "r"(hi.w)
                             : "memory");
            }
        }
    } else {
        const bool in_row = dim < a.D;
#pragma unroll 4
        for (int k = lane / kUnits; k < kKeys; k += kStep) {
            const long long r = row_of(key0 + k);
            const uint16_t *src = r < 0 ? a.win + (size_t)~r * a.D + dim : a.kv + (size_t)r * a.D + dim;
            cp_async16_or_zero(at(k, u), r != kNone && in_row ? src : nullptr, a.win);
        }
    }
}

template <int DP, bool FP8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attend_prefix_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const Params p) {
    using Lt = Layout<DP>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const Smem s = carve<DP>(smem_raw);
    const AttendArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_rank(), pair = blockIdx.x >> 1;
    const bool q_rw = a.q_gain != nullptr || a.rope_cos != nullptr;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kSlots; ++i) {
            mbar_init(s.full + i, 2);   // used on the leader: each CTA's producer (+ bytes of both)
            mbar_init(s.empty + i, 1);  // commit
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s.sfull + i, 1);
            mbar_init(s.sempty + i, 2 * kSoftWarps);  // leader: the softmax warps of both CTAs
            mbar_init(s.pfull + i, 2 * kSoftWarps);   // leader
            mbar_init(s.pvdone + i, 1);
        }
        mbar_init(s.qland, 1);
        mbar_init(s.qready, q_rw ? 2 * kSoftWarps : 2);  // leader
        mbar_init(s.qempty, 1 + kSoftWarps);
        for (int i = 0; i < 2; ++i) mbar_init(s.vfix + i, 1);
        for (int i = 0; i < kDescs; ++i) {
            mbar_init(s.dfull + i, 1);
            mbar_init(s.dempty + i, kSoftWarps + 1);  // and the query tiles' warp
        }
        *s.abort_flag = 0;
        fence_mbar_init();
        tc::prefetch_tmap(&qmap);
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
    }
    if (warp == kQueryWarp) tc::tmem_alloc_2sm(smem_u32(s.tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();  // both CTAs' barriers exist
    tc::fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = *s.tmem_slot;

    // tile number g's description, once it is there (null: given up)
    const auto desc_of = [&](uint32_t g) -> const Tile * {
        return mbar_wait(smem_u32(s.dfull + g % kDescs), (g / kDescs) & 1u, p.ctx, s.abort_flag) ? s.desc + g % kDescs
                                                                                                 : nullptr;
    };
    const auto warp_desc_of = [&](uint32_t g) -> const Tile * {
        const Tile *d = desc_of(g);
        return __all_sync(0xffffffffu, d != nullptr) ? d : nullptr;
    };
    bool copies = false;  // given up with TMA copies in flight, maybe

    if (warp < kProducers) {
        // ------------------------------------------------------------ producers
        // The copies of an own slot are in flight while the warp's next slot is issued (unless
        // that one is not free yet).  TMA copies are issued by one thread inside an elect_one
        // branch (one issued by every lane under a guard, or by a diverged lane, took ~200
        // cycles: more than the MMAs that it feeds).
        if (p.linear) asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows' copy
        const bool v = warp >= 2;  // K's or V's ring
        const int ring = v ? kSlots : 0;
        const uint32_t full0 = tc::map_to_rank(smem_u32(s.full + ring), 0), slots = smem_u32(s.slots) + ring * kSlotBytes;
        const uint32_t vfix = smem_u32(s.vfix + (warp & 1));
        uint32_t it = 0, nfix = 0;  // ring position
        int pending = -1;
        bool ok = true;
        const auto flush = [&] {
            if (pending < 0) return;
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            tc::fence_proxy_async_smem();
            __syncwarp();
            mbar_arrive_cluster(full0 + pending * 8, lane == 0);
            pending = -1;
        };
        for (uint32_t g = 0; ok; ++g) {
            const Tile *dp = warp_desc_of(g);
            if (!(ok = dp != nullptr)) break;
            const Tile &d = *dp;
            if (d.flags & kEnd) break;
#pragma unroll 1
            for (int w = 0; w < Lt::kPieces && ok; ++w, ++it) {
                if ((it ^ (uint32_t)warp) & 1u) continue;
                const uint32_t sl = it % kSlots, par = ((it / kSlots) & 1u) ^ 1u, empty = smem_u32(s.empty + ring + sl);
                const uint32_t dst = slots + sl * kSlotBytes, full = full0 + sl * 8;
                if (!__all_sync(0xffffffffu, mbar_test_wait(empty, par))) {
                    flush();
                    if (!(ok = warp_wait(empty, par, p.ctx, s.abort_flag))) break;
                }
                if (!(d.flags & kShared)) {
                    if (v) gather_slot<DP, FP8, true>(p, d, rank, w, dst);
                    else gather_slot<DP, FP8, false>(p, d, rank, w, dst);
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    const int before = pending;
                    pending = (int)sl;
                    if (FP8) {
                        flush();
                    } else if (before >= 0) {
                        asm volatile("cp.async.wait_group 1;" ::: "memory");
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        mbar_arrive_cluster(full0 + before * 8, lane == 0);
                    }
                    continue;
                }
                flush();
                if (!v) {
                    if (tc::elect_one()) {
                        mbar_arrive_expect_tx_cluster(full, kSlotBytes);
                        if (p.box == 64) {
                            tc::tma_load_3d_2sm(dst, &kmap, full, 0, d.rows[rank * 4], 2 * w);
                        } else {
                            for (int x = 0; x < 64; x += p.box) {
                                const int row = d.rows[rank * 4 + x / 16];
                                tc::tma_load_3d_2sm(dst + x * 128, &kmap, full, 0, row, 2 * w);
                                tc::tma_load_3d_2sm(dst + 8192 + x * 128, &kmap, full, 0, row, 2 * w + 1);
                            }
                        }
                    }
                    __syncwarp();
                    continue;
                }
                // V: entries of the tile that do not count have zero weights; their values (anything,
                // in memory) are cleared where a copy brings them
                const int end = d.ent - w * Lt::kVKeys;  // entries of the slot that count
                const bool fix = end > 0 && end < Lt::kVKeys && (end & (p.vbox - 1)) != 0;
                if (tc::elect_one()) {
                    const uint32_t bar = fix ? tc::map_to_rank(vfix, rank) : full;
                    mbar_arrive_expect_tx_cluster(bar, kSlotBytes);
                    for (int x = 0; x < Lt::kVKeys; x += p.vbox)
                        tc::tma_load_3d_2sm(dst + x * (Lt::kVChunks * 128), &vmap, bar, 0, d.rows[(w * Lt::kVKeys + x) / 16],
                                            rank * Lt::kVChunks);
                }
                __syncwarp();
                if (fix) {
                    if (!(ok = warp_wait(vfix, nfix & 1u, p.ctx, s.abort_flag))) break;
                    ++nfix;
                    // entry e of the slot, chunk c: [e / vbox][c][e % vbox][128 B]
                    uint4 *slot = reinterpret_cast<uint4 *>(s.slots + (ring + sl) * kSlotBytes);
#pragma unroll 1
                    for (int y = lane; y < Lt::kVKeys * Lt::kVChunks * 8; y += 32) {
                        const int line = y >> 3, e = line / (Lt::kVChunks * p.vbox) * p.vbox + (line & (p.vbox - 1));
                        if (e >= end) slot[y] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    mbar_arrive_cluster(full, lane == 0);
                }
            }
        }
        if (ok) flush();
        asm volatile("cp.async.wait_all;" ::: "memory");
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
                const uint32_t b = g & 1u;
                if (flags & kFirst) {
                    if (!mbar_wait(smem_u32(s.qready), nq & 1u, p.ctx, s.abort_flag)) break;
                    ++nq;
                }
                if (!mbar_wait(smem_u32(s.sempty + b), ((g >> 1) & 1u) ^ 1u, p.ctx, s.abort_flag)) break;
                for (int w = 0; w < Lt::kPieces; ++w, ++it) {
                    const uint32_t sl = it % kSlots;
                    if (!(ok = mbar_wait(smem_u32(s.full + sl), (it / kSlots) & 1u, p.ctx, s.abort_flag))) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // 16 dims each: chunk 2 w + k / 4
                        const uint32_t off = (k >> 2) * 8192 + (k & 3) * 32;
                        tc::mma_f16_2sm(tmem + kSCols + b * 64, qdesc + ((w * 16384 + off) >> 4),
                                        kdesc + ((sl * kSlotBytes + off) >> 4), p.idesc_qk, (w | k) ? 1u : 0u);
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
            const uint64_t vdesc =
                tc::smem_desc_lbo(smem_u32(s.slots) + kSlots * kSlotBytes, p.vbox * 128, 1024, tc::kLayoutSw128);
            const uint64_t pdesc = tc::smem_desc(smem_u32(s.p), 1024, tc::kLayoutSw128);
            const int vsh = 31 - __clz(p.vbox);
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t g = 0; ok; ++g) {
                const Tile *d = desc_of(g);
                if (!d) break;
                const int flags = d->flags;
                if (flags & kEnd) break;
                const uint32_t b = g & 1u;
                if (!mbar_wait(smem_u32(s.pfull + b), (g >> 1) & 1u, p.ctx, s.abort_flag)) break;
                for (int w = 0; w < Lt::kPieces; ++w, ++it) {
                    const uint32_t sl = it % kSlots;
                    if (!(ok = mbar_wait(smem_u32(s.full + kSlots + sl), (it / kSlots) & 1u, p.ctx, s.abort_flag))) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int k = 0; k < Lt::kVKeys / 16; ++k) {  // 16 keys each
                        const uint32_t kt = w * (Lt::kVKeys / 16) + k, x = k * 16;
                        const uint32_t voff = ((((x >> vsh) * Lt::kVChunks) << vsh) + (x & (p.vbox - 1))) * 128;
#pragma unroll
                        for (int i = 0; i < Lt::kPvMmas; ++i)
                            tc::mma_f16_2sm(tmem + i * (Lt::kPvN / 2),
                                            pdesc + ((b * kPBytes + (kt >> 2) * 8192 + (kt & 3) * 32) >> 4),
                                            vdesc + ((sl * kSlotBytes + voff + i * 2 * p.vbox * 128) >> 4), p.idesc_pv,
                                            (!(flags & kFirst) || kt) ? 1u : 0u);
                    }
                    tc::mma_commit_2sm(smem_u32(s.empty + kSlots + sl));
                }
                if (!ok) break;
                tc::mma_commit_2sm(smem_u32(s.pvdone + b));
            }
        }
    } else if (warp == kQueryWarp) {
        // ------------------------------------------------------------ query tiles
        const uint32_t qland = tc::map_to_rank(smem_u32(s.qland), rank), qready0 = tc::map_to_rank(smem_u32(s.qready), 0);
        uint32_t nq = 0;
        bool ok = true;
        for (uint32_t g = 0; ok; ++g) {
            const Tile *d = warp_desc_of(g);
            if (!(ok = d != nullptr)) break;
            const int flags = d->flags, row = d->rt * kPrefixRows + rank * 64;
            __syncwarp();
            mbar_arrive(smem_u32(s.dempty + g % kDescs), lane == 0);
            if (flags & kEnd) break;
            if (!(flags & kFirst)) continue;
            if (!(ok = warp_wait(smem_u32(s.qempty), (nq & 1u) ^ 1u, p.ctx, s.abort_flag))) break;
            if (tc::elect_one()) {
                mbar_arrive_expect_tx_cluster(qland, Lt::kQBytes);
                for (int c = 0; c < DP / 64; c += 2)
                    tc::tma_load_3d_2sm(smem_u32(s.q) + c * 8192, &qmap, qland, 0, row, c);
            }
            __syncwarp();
            if (!(ok = warp_wait(smem_u32(s.qland), nq & 1u, p.ctx, s.abort_flag))) break;
            if (!q_rw) mbar_arrive_cluster(qready0, lane == 0);  // else the softmax warps rewrite the tile first
            ++nq;
        }
        copies = !ok;
    } else if (warp == kPlanWarp) {
        // ------------------------------------------------------------ planner
        Units un = deal_units(p, pair, blockIdx.x == 0);
        uint32_t g = 0;
        bool ok = true;
        // An entry is free for tile g once tile g - kDescs is done with everywhere: once the
        // softmax warps are done with tile g - kDescs + 2, whose P went where the P of that tile was.
        const auto entry = [&]() -> Tile * {
            const int h = (int)g - kDescs + 2;
            if (h >= 0) ok = warp_wait(smem_u32(s.dempty + h % kDescs), (uint32_t)(h / kDescs) & 1u, p.ctx, s.abort_flag);
            return ok ? s.desc + g % kDescs : nullptr;
        };
        const auto publish = [&] {
            __syncwarp();
            mbar_arrive(smem_u32(s.dfull + g % kDescs), lane == 0);
            ++g;
        };
        while (un.left > 0 && ok) {
            const Queries qs = queries_of(p, un.rt);
            const int b0 = qs.bq0 / a.nq, b1 = qs.bq1 / a.nq;
            int vmax = 0, n = 0;
            for (int q = qs.bq0 + lane; q <= qs.bq1; q += 32) vmax = std::max(vmax, visible(p, __ldg(a.q_pos + q), p.n_shared));
            const auto request = [&](int b) {
                return own_keys(p, std::max(qs.bq0, b * a.nq), std::min(qs.bq1, b * a.nq + a.nq - 1));
            };
            for (int b = b0 + lane; b <= b1; b += 32) n += request(b).tiles();
            vmax = __reduce_max_sync(0xffffffffu, vmax);
            const int shared = (vmax + kPrefixKeys - 1) / kPrefixKeys;
            n = __reduce_add_sync(0xffffffffu, n) + shared - un.x;
            if (n > 0) {
                n = (int)std::min<long long>(n, un.left);
                un.left -= n;
                int x = un.x, b = b0 - 1;
                long long y = x - shared;  // the tile's number among its request's own ones
                Own own = {0, 0, 0};
                for (int j = 0; j < n && ok; ++j, ++x, ++y) {
                    Tile *d = entry();
                    if (!d) break;
                    const bool sh = x < shared;
                    int ent, cnt, e_first, wpos = 0, ring = 0;
                    if (sh) {
                        e_first = x * kPrefixKeys;
                        cnt = ent = std::min(vmax - e_first, +kPrefixKeys);
                    } else {
                        while (y >= own.tiles()) {
                            y -= own.tiles();
                            own = request(++b);
                        }
                        const long long first = y * kPrefixKeys;
                        e_first = (int)std::min<long long>(p.n_shared + first, 0x7fffffff);
                        ent = (int)std::min<long long>(std::max<long long>(own.n_own - first, 0), +kPrefixKeys);
                        cnt = (int)std::min<long long>(own.total - first, +kPrefixKeys);
                        wpos = (int)(own.u0 + first - own.n_own);
                        ring = ent < cnt ? (int)((uint32_t)(wpos + ent) % (uint32_t)a.win_rows) : 0;
                    }
                    int row = -kPrefixKeys;
                    bool missing = false;
                    if (lane < 8 && lane * 16 < ent) {
                        const uint32_t e = (uint32_t)(e_first + lane * 16), pg = e / (uint32_t)a.page;
                        const int id = __ldg(a.table + (sh ? 0 : (size_t)b * a.max_pages) + pg);
                        missing = id < 0 || id >= a.n_pages;
                        if (sh && p.linear) row = (int)e;
                        else if (!missing) row = id * a.page + (int)(e - pg * (uint32_t)a.page);
                    }
                    if (lane < 8) d->rows[lane] = row;
                    const int miss = (int)__ballot_sync(0xffffffffu, missing);
                    if (lane == 0) {
                        d->flags = (sh ? kShared : 0) | (j == 0 ? kFirst : 0) | (j == n - 1 ? kLast : 0) | (miss << kMissingShift);
                        d->rt = un.rt;
                        d->b = b;
                        d->e_first = e_first;
                        d->ent = ent;
                        d->cnt = cnt;
                        d->wpos = wpos;
                        d->ring = ring;
                    }
                    publish();
                    if (sh || rank == 0) continue;
                    // own rows into L2, by the pair's other CTA
#pragma unroll 1
                    for (int k = lane; k < kPrefixKeys; k += 32) {
                        const int er = __shfl_sync(0xffffffffu, row, k >> 4);
                        const void *src = nullptr;
                        if (k < ent) {
                            if (er >= 0) src = FP8 ? (const void *)(a.kv8 + (size_t)(er + (k & 15)) * a.D)
                                                   : (const void *)(a.kv + (size_t)(er + (k & 15)) * a.D);
                        } else if (k < cnt) {
                            const size_t r = (size_t)b * a.win_rows + (uint32_t)(wpos + k) % (uint32_t)a.win_rows;
                            src = FP8 ? (const void *)(a.win8 + r * a.D) : (const void *)(a.win + r * a.D);
                        }
                        if (src)
                            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(FP8 ? a.D : 2 * a.D)
                                         : "memory");
                    }
                }
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
    } else {
        // ------------------------------------------------------------ softmax, partial rows
        // The four warps of 32 rows meet at named barriers: a wait that was given up is told to
        // all of them at the next one (group_all), so that they leave together.
        const int quarter = warp & 3, wg = (warp - kSoftWarp0) >> 2;
        const int tl = quarter * 32 + lane;       // tensor-memory lane
        const int r = tl & 63, hf = tl >> 6;      // row of this CTA's 64; first / second half of the columns
        const int q4 = hf * 2 + wg;               // which of the row's four threads
        const int off = hf * 64 + wg * 32;        // its first key of a tile
        const int bar_id = 1 + (quarter & 1);     // the 128 threads of 32 rows
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t sempty0 = tc::map_to_rank(smem_u32(s.sempty), 0), pfull0 = tc::map_to_rank(smem_u32(s.pfull), 0);
        const uint32_t qready0 = tc::map_to_rank(smem_u32(s.qready), 0);
        const int n_rows = (int)(a.n_bq * a.H);
        uint32_t nq = 0;
        int t = -1, vis = 0, b_row = 0;
        float rq = 0.f, m_run = -INFINITY, l = 0.f;
        const Tile *d = warp_desc_of(0);
        bool ok = group_all(bar_id, d != nullptr);
        if (!ok) d = nullptr;
        for (uint32_t g = 0; d; ++g) {
            const int flags = d->flags;
            if (flags & kEnd) break;
            const uint32_t b = g & 1u, ph = (g >> 1) & 1u;
            if (flags & kFirst) {  // a new row tile
                const int row = d->rt * kPrefixRows + rank * 64 + r;
                const int bq = row < n_rows ? row / a.H : 0;
                t = row < n_rows ? __ldg(a.q_pos + bq) : -1;
                b_row = bq / a.nq;
                vis = visible(p, t, (int)a.N);
                ok = warp_wait(smem_u32(s.qland), nq & 1u, p.ctx, s.abort_flag);
                ++nq;
                s.xsum[q4 * 64 + r] = query_squares<DP>(s.q, r, q4);
                if (q_rw) {
                    query_rewrite<DP>(a, s.q, r, q4, t);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    mbar_arrive_cluster(qready0, lane == 0);
                }
                __syncwarp();
                mbar_arrive(smem_u32(s.qempty), lane == 0);
                group_sync(bar_id);
                const float ss = (s.xsum[r] + s.xsum[64 + r]) + (s.xsum[128 + r] + s.xsum[192 + r]);
                group_sync(bar_id);
                // 1 / RMS times the softmax scale, in log2 units
                rq = (1.0f / sqrtf(ss / (float)a.D + a.eps)) * a.scale * 1.4426950408889634f;
                m_run = -INFINITY;
                l = 0.f;
            }
            const uint32_t mask = key_mask(*d, off, t, a.W, vis, b_row);  // keys that take part
            const bool whole = __all_sync(0xffffffffu, mask == 0xffffffffu);
            const size_t part = (size_t)pair + d->rt;
            const Tile *next = warp_desc_of(g + 1);
            ok = warp_wait(smem_u32(s.sfull + b), ph, p.ctx, s.abort_flag) && next && ok;
            tc::fence_after_sync();
            float sc[32];
            tc::tmem_ld32(tmem + lane_base + kSCols + b * 64 + wg * 32, sc);
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            __syncwarp();
            mbar_arrive_cluster(sempty0 + b * 8, lane == 0);
            // the largest scaled score: the largest raw one, or the smallest under a negative scale
            float mt = -INFINITY;
            if (whole && rq >= 0.f) {
                float m2 = sc[1];
                mt = sc[0];
#pragma unroll
                for (int i = 2; i < 32; i += 2) {
                    mt = fmaxf(mt, sc[i]);
                    m2 = fmaxf(m2, sc[i + 1]);
                }
                mt = fmaxf(mt, m2) * rq;
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) mt = fmaxf(mt, (mask >> i) & 1u ? sc[i] * rq : -INFINITY);
            }
            // the row's maximum over its four threads, each rounded to 16 bits towards zero
            // (any reference near the maximum serves, as long as the four agree)
            s.xmax[(b * 4 + q4) * 64 + r] = (uint16_t)(__float_as_uint(mt) >> 16);
            if (!group_all(bar_id, ok)) break;
            mt = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) mt = fmaxf(mt, __uint_as_float((uint32_t)s.xmax[(b * 4 + i) * 64 + r] << 16));
            const bool mine = m_run != -INFINITY && mt > m_run + kRescaleThreshold;
            if (__any_sync(0xffffffffu, mine)) {
                const uint32_t gp = g - 1;  // O after the P.V of the tile before
                ok = warp_wait(smem_u32(s.pvdone + (gp & 1u)), (gp >> 1) & 1u, p.ctx, s.abort_flag) && ok;
                tc::fence_after_sync();
                const float f = mine ? exp2f(m_run - mt) : 1.0f;
#pragma unroll 1
                for (int c = wg * (DP / 4); c < (wg + 1) * (DP / 4); c += 16) {
                    float v[16];
                    tc::tmem_ld16(tmem + lane_base + c, v);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] *= f;
                    tc::tmem_st16(tmem + lane_base + c, v);
                }
                tc::tmem_wait_st();
                if (mine) {
                    l *= f;
                    m_run = mt;
                }
            }
            if (m_run == -INFINITY) m_run = mt;
            const float mref = m_run == -INFINITY ? 0.f : m_run;
            float ps[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 32; ++i) sc[i] = exp2_ftz(fmaf(sc[i], rq, -mref));
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 32; ++i) sc[i] = (mask >> i) & 1u ? sc[i] : 0.f;
            }
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                ps[0] += sc[i];
                ps[1] += sc[i + 1];
                pk[i / 2] = pack_bf16x2(sc[i], sc[i + 1]);
            }
            l += ps[0] + ps[1];
            // P buffer b was read by the P.V of tile g - 2
            ok = warp_wait(smem_u32(s.pvdone + b), ph ^ 1u, p.ctx, s.abort_flag) && ok;
            uint8_t *prow = s.p + b * kPBytes + hf * 8192 + r * 128;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint4 *>(prow + (((wg * 4 + x) ^ (r & 7)) << 4)) =
                    make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
            tc::fence_proxy_async_smem();
            tc::fence_before_sync();
            __syncwarp();
            mbar_arrive_cluster(pfull0 + b * 8, lane == 0);
            mbar_arrive(smem_u32(s.dempty + g % kDescs), lane == 0);
            if (flags & kLast) {
                ok = warp_wait(smem_u32(s.pvdone + b), ph, p.ctx, s.abort_flag) && ok;
                tc::fence_after_sync();
                s.xsum[q4 * 64 + r] = l;  // (every thread has read the last tile's maxima)
                group_sync(bar_id);
                if (q4 == 0)
                    p.ml[part * kPrefixRows + rank * 64 + r] =
                        make_float2(m_run, (s.xsum[r] + s.xsum[64 + r]) + (s.xsum[128 + r] + s.xsum[192 + r]));
                group_sync(bar_id);
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
            }
            d = next;
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

// Rows 0..n_shared-1 of an FP8 pool in order, as bf16 (exact); entries without a page are zero.
__global__ void __launch_bounds__(256)
    prefix_rows_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ exps, const int *__restrict__ table,
                       int page, long long n_pages, int D, long long units, uint4 *__restrict__ out) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long u = (long long)blockIdx.x * 256 + threadIdx.x;  // 16 codes each
    if (u >= units) return;
    const int upr = D / 16;
    const uint32_t j = (uint32_t)(u / upr);
    const int c = (int)(u - (long long)j * upr);
    const int id = __ldg(table + j / (uint32_t)page);
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (id >= 0 && id < n_pages) {
        const size_t row = (size_t)id * page + j % (uint32_t)page;
        const uint4 v = ldg_stream(codes + row * D + c * 16);
        const uint32_t e = __ldg(exps + row * (D / 128) + c / 8);
        lo = e4m3x8_bf16x8(make_uint2(v.x, v.y), e);
        hi = e4m3x8_bf16x8(make_uint2(v.z, v.w), e);
    }
    out[2 * u] = lo;
    out[2 * u + 1] = hi;
}

// kind::f16 instruction descriptor: bf16 operands, fp32 accumulate, M = 128
constexpr uint32_t idesc(int n, bool b_mn) { return tc::idesc_f16(n, true) | (b_mn ? (1u << 16) : 0u); }

template <int DP, bool FP8>
int launch_d(const PrefixArgs &x, const DevCtx &ctx, cudaStream_t st) {
    Params p = {};
    p.a = x.a;
    p.plan = x.plan;
    p.n_shared = (int)x.n_shared;
    p.linear = x.linear ? 1 : 0;
    p.part = x.part;
    p.ml = x.ml;
    p.first = x.first;
    p.ctx = ctx;
    p.idesc_qk = idesc(kPrefixKeys, false);
    p.idesc_pv = idesc(Layout<DP>::kPvN, true);
    p.box = x.linear || x.a.page % 64 == 0 ? 64 : (x.a.page % 32 == 0 ? 32 : 16);
    p.vbox = std::min(p.box, Layout<DP>::kVKeys);
    auto kern = attend_prefix_kernel<DP, FP8>;
    constexpr size_t smem = smem_bytes<DP>();
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return CSA_ERR_CUDA;
    // [64-dim chunk][row][64]: one copy brings several chunks of its rows (past D: zeros)
    const auto encode = [&](CUtensorMap *map, const uint16_t *base, long long rows, int box_rows, int chunks) {
        const uint64_t dims[3] = {64, (uint64_t)rows, (uint64_t)(x.a.D / 64)};
        const uint64_t strides[2] = {(uint64_t)x.a.D * 2, 128};
        const uint32_t box[3] = {64, (uint32_t)box_rows, (uint32_t)chunks};
        return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                                 CU_TENSOR_MAP_SWIZZLE_128B);
    };
    const long long key_rows = x.linear ? x.n_shared : x.a.n_pages * x.a.page;
    CUtensorMap qmap, kmap, vmap;
    if (!encode(&qmap, x.a.q, x.a.n_bq * x.a.H, 64, 2) || !encode(&kmap, x.keys, key_rows, p.box, p.box == 64 ? 2 : 1) ||
        !encode(&vmap, x.keys, key_rows, p.vbox, Layout<DP>::kVChunks))
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
    cfg.numAttrs = x.linear ? 1 : 0;  // a dependent of the rows' copy
    return cudaLaunchKernelEx(&cfg, kern, qmap, kmap, vmap, p) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // namespace

PrefixPlan prefix_plan(long long rows) {
    PrefixPlan pl;
    pl.row_tiles = (int)((rows + kPrefixRows - 1) / kPrefixRows);
    pl.pairs = std::max(num_sms() / 2, 1);
    return pl;
}

int launch_prefix_rows(const uint8_t *codes, const uint8_t *exps, const int *table, int page, long long n_pages, int D,
                       long long n_shared, uint16_t *out, cudaStream_t st) {
    const long long units = n_shared * (D / 16), blocks = (units + 255) / 256;
    prefix_rows_kernel<<<(unsigned)blocks, 256, 0, st>>>(codes, exps, table, page, n_pages, D, units,
                                                         reinterpret_cast<uint4 *>(out));
    return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

int launch_attend_prefix(const PrefixArgs &p, const DevCtx &ctx, cudaStream_t st) {
    const bool fp8 = p.a.kv8 != nullptr;
    switch (prefix_dims(p.a.D)) {
        case 128: return fp8 ? launch_d<128, true>(p, ctx, st) : launch_d<128, false>(p, ctx, st);
        case 256: return fp8 ? launch_d<256, true>(p, ctx, st) : launch_d<256, false>(p, ctx, st);
        case 512: return fp8 ? launch_d<512, true>(p, ctx, st) : launch_d<512, false>(p, ctx, st);
        default: return CSA_ERR_UNSUPPORTED;
    }
}

}  // namespace csa
