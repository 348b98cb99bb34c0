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
// Warps: 0..3 producers of K and V, 4 MMA issuer (the pair's leader), 5 tensor
// memory and the query tile, 6..13 softmax (four threads per row: lane half x
// 32-column half).  16 KiB slots form one ring for both operands, in the order
// the MMAs consume them (K0, K1, V0, K2, V1, ...); the producers take its
// positions in turn, whatever they hold: shared entries by TMA, own keys (rows
// of any page and of the ring) by 16-byte asynchronous copies, FP8 rows expanded
// on the way.  (A producer per kind would pass over the other kind's positions,
// and a slot's phase bit cannot tell it how far the ring is.)
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

constexpr int kThreads = 448;
constexpr int kProducers = 4, kMmaWarp = 4, kQueryWarp = 5, kSoftWarp0 = 6, kSoftWarps = 8;
constexpr int kSlots = 8;
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

struct Smem {
    uint8_t *q, *slots, *p;
    uint64_t *full, *empty, *sfull, *sempty, *pfull, *pvdone, *qland, *qready, *qempty, *vfix;
    uint16_t *xmax;  // [2][4][64] the upper halves of the row maxima of a tile's four threads per row
    float *xsum;     // [4][64], the same memory
    long long *left; // this pair's units
    int *start;      // its first row tile, and the first unit's number within it
    uint32_t *tmem_slot;
    int *abort_flag;
};

template <int DP>
CSA_DEVINL Smem carve(uint8_t *raw) {
    Smem s;
    s.q = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    s.slots = s.q + Layout<DP>::kQBytes;
    s.p = s.slots + kSlots * kSlotBytes;
    s.xsum = reinterpret_cast<float *>(s.p + 2 * kPBytes);
    s.xmax = reinterpret_cast<uint16_t *>(s.xsum);
    uint64_t *bars = reinterpret_cast<uint64_t *>(s.xsum + 256);
    s.full = bars;
    s.empty = bars + kSlots;
    s.sfull = bars + 2 * kSlots;
    s.sempty = s.sfull + 2;
    s.pfull = s.sempty + 2;
    s.pvdone = s.pfull + 2;
    s.qland = s.pvdone + 2;
    s.qready = s.qland + 1;
    s.qempty = s.qready + 1;
    s.vfix = s.qempty + 1;
    s.left = reinterpret_cast<long long *>(s.vfix + kProducers);
    s.start = reinterpret_cast<int *>(s.left + 1);
    s.tmem_slot = reinterpret_cast<uint32_t *>(s.start + 2);
    s.abort_flag = reinterpret_cast<int *>(s.tmem_slot + 1);
    return s;
}

template <int DP>
constexpr size_t smem_bytes() {
    return 1024 + Layout<DP>::kQBytes + kSlots * kSlotBytes + 2 * kPBytes + 1024 + (2 * kSlots + 11 + kProducers) * 8 + 32;
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

// units of row tile rt, by one thread
CSA_DEVINL int count_units(const Params &p, int rt) {
    const Queries r = queries_of(p, rt);
    int vmax = 0, n = 0;
    for (int q = r.bq0; q <= r.bq1;) {
        const int e = std::min(r.bq1, q / p.a.nq * p.a.nq + p.a.nq - 1);
        n += own_keys(p, q, e).tiles();
        for (; q <= e; ++q) vmax = std::max(vmax, visible(p, __ldg(p.a.q_pos + q), p.n_shared));
    }
    return n + (vmax + kPrefixKeys - 1) / kPrefixKeys;
}

// Which units are this pair's, by one warp; pair 0 writes where the row tiles begin.
CSA_DEVINL void deal_units(const Params &p, const Smem &s, int pair, bool write) {
    const int lane = threadIdx.x & 31, RT = p.plan.row_tiles;
    long long total = 0;
    int n = 0;
    for (int r0 = 0; r0 < RT; r0 += 32) {
        n = r0 + lane < RT ? count_units(p, r0 + lane) : 0;
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += up;
        }
        if (write && r0 + lane < RT) p.first[r0 + lane] = total + inc - n;
        total += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (write && lane == 0) p.first[RT] = total;
    const int P = p.plan.active(total);
    const long long u0 = pair < P ? total * pair / P : 0, u1 = pair < P ? total * (pair + 1) / P : 0;
    if (lane == 0) *s.left = u1 - u0;
    if (u1 == u0) return;
    long long base = 0;
    for (int r0 = 0; r0 < RT; r0 += 32) {
        if (RT > 32) n = r0 + lane < RT ? count_units(p, r0 + lane) : 0;
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += up;
        }
        if (base + inc - n <= u0 && u0 < base + inc) {
            s.start[0] = r0 + lane;
            s.start[1] = (int)(u0 - (base + inc - n));
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
        if (base > u0) break;
    }
}

// A pair's part of one row tile: n of its tiles from number x on.
struct Range {
    int rt, x, n;
    int vmax, shared;  // shared entries that any of its rows sees, and their tiles
    Queries q;
};

// One of a range's tiles: 128 shared entries (own.total < 0) or packed own keys, from `first` on.
struct Tile {
    long long first;
    int b;  // the request
    Own own;
    CSA_DEVINL bool shared() const { return own.total < 0; }
};

// Walks a pair's ranges and the tiles of each; every role does so by itself, whole warps together.
struct Walk {
    long long left;
    int rt, x;
    CSA_DEVINL explicit Walk(const Smem &s) : left(*s.left), rt(s.start[0]), x(s.start[1]) {}

    CSA_DEVINL bool next(const Params &p, Range &r) {
        const int lane = threadIdx.x & 31;
        while (left > 0) {
            r.rt = rt;
            r.x = x;
            r.q = queries_of(p, rt);
            int v = 0, n = 0;
            for (int q = r.q.bq0 + lane; q <= r.q.bq1; q += 32) v = std::max(v, visible(p, __ldg(p.a.q_pos + q), p.n_shared));
            const int b0 = r.q.bq0 / p.a.nq, b1 = r.q.bq1 / p.a.nq;
            for (int b = b0 + lane; b <= b1; b += 32)
                n += own_keys(p, std::max(r.q.bq0, b * p.a.nq), std::min(r.q.bq1, b * p.a.nq + p.a.nq - 1)).tiles();
            r.vmax = __reduce_max_sync(0xffffffffu, v);
            r.shared = (r.vmax + kPrefixKeys - 1) / kPrefixKeys;
            n = __reduce_add_sync(0xffffffffu, n) + r.shared - x;
            ++rt;
            x = 0;
            if (n <= 0) continue;
            r.n = (int)std::min<long long>(n, left);
            left -= r.n;
            return true;
        }
        return false;
    }
};

struct Tiles {
    Tile t;
    int x;

    CSA_DEVINL void request(const Params &p, const Range &r, int b) {
        t.b = b;
        t.own = own_keys(p, std::max(r.q.bq0, b * p.a.nq), std::min(r.q.bq1, b * p.a.nq + p.a.nq - 1));
    }
    CSA_DEVINL Tiles(const Params &p, const Range &r) {
        x = r.x;
        t.own.total = -1;
        t.own.n_own = t.own.u0 = t.b = 0;
        t.first = (long long)x * kPrefixKeys;
        if (x >= r.shared) {
            long long y = x - r.shared;
            request(p, r, r.q.bq0 / p.a.nq);
            while (y >= t.own.tiles()) {
                y -= t.own.tiles();
                request(p, r, t.b + 1);
            }
            t.first = y * kPrefixKeys;
        }
    }
    CSA_DEVINL void next(const Params &p, const Range &r) {
        ++x;
        t.first += kPrefixKeys;
        if (x < r.shared) return;
        if (x == r.shared) {
            t.first = 0;
            request(p, r, r.q.bq0 / p.a.nq);
        }
        while (t.first >= t.own.total) {
            t.first = 0;
            request(p, r, t.b + 1);
        }
    }
};

CSA_DEVINL bool warp_wait(uint32_t bar, uint32_t parity, const DevCtx &ctx, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctx, abort));
}

CSA_DEVINL void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// The tile's query rows as they landed: this thread's quarter of row r (units
// q4, q4 + 4, .. of 8 dims) -> its sum of squares; with a gain or RoPE the
// units are rewritten (gain, then the rotation of the trailing kRopeDim
// channels: unit j of the slice pairs with j + 4, also this thread's), rounded
// to bf16 as the tensor cores' operand.
template <int DP>
CSA_DEVINL float query_units(const AttendArgs &a, uint8_t *q, int r, int q4, long long t, bool rewrite) {
    float ss = 0.f;
    const int r0 = a.D / 8 - kRopeDim / 8;  // first rotated unit
#pragma unroll
    for (int i = 0; i < DP / 32; i += 2) {
        uint4 *ptr[2];
        float x[2][8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int unit = q4 + 4 * (i + k);
            ptr[k] = reinterpret_cast<uint4 *>(q + (unit >> 3) * 8192 + r * 128 + (((unit & 7) ^ (r & 7)) << 4));
            unpack8(*ptr[k], x[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[k][e], x[k][e], ss);
        }
        if (rewrite) {
            const int unit = q4 + 4 * i;
            if (unit * 8 < a.D) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (a.q_gain) x[k][e] *= __ldg(a.q_gain + (unit + 4 * k) * 8 + e);
                if (a.rope_cos && unit >= r0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 cs = rope_cs(a, t, (unit - r0) * 8 + e);
                        const float x0 = x[0][e], x1 = x[1][e];
                        x[0][e] = x0 * cs.x - x1 * cs.y;
                        x[1][e] = x1 * cs.x + x0 * cs.y;
                    }
                }
                *ptr[0] = pack8(x[0]);
                *ptr[1] = pack8(x[1]);
            }
        }
    }
    return ss;
}

CSA_DEVINL uint32_t low_bits(long long n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << (int)n) - 1u); }

// Which of keys off..off + 31 of a tile the row of a query at t (of request
// b_row, seeing vis shared entries) takes.
CSA_DEVINL uint32_t key_mask(const Params &p, const Tile &tile, int off, int t, int vis, int b_row) {
    const AttendArgs &a = p.a;
    const long long k0 = tile.first + off;  // entry, or packed own key
    const int *table = a.table;
    long long ent, e0 = k0;  // entries from e0 on: the first `ent` of the 32 keys are the row's
    uint32_t mask;
    if (tile.shared()) {
        ent = vis - k0;
        mask = low_bits(ent);
    } else {
        if (t < 0 || b_row != tile.b) return 0u;
        ent = std::max(0, visible(p, t, (int)a.N) - p.n_shared) - k0;
        // positions t-W+1..t, key n_own + (u - u0)
        const long long lo = tile.own.n_own + (long long)std::max(0, t - a.W + 1) - tile.own.u0 - k0;
        const long long hi = tile.own.n_own + (long long)t - tile.own.u0 - k0;
        mask = low_bits(ent) | (low_bits(hi + 1) & ~low_bits(lo));
        table += (size_t)tile.b * a.max_pages;
        e0 += p.n_shared;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (ent > 16 * h) {  // 16 entries of one page (n_shared, k0 and the page are multiples of 16)
            const int id = __ldg(table + (uint32_t)(e0 + 16 * h) / (uint32_t)a.page);
            if (id < 0 || id >= a.n_pages) mask &= ~(low_bits(std::min(ent - 16 * h, 16LL)) << (16 * h));
        }
    return mask;
}

// One slot of an own tile, by one warp: K (V = false): the CTA's 64 keys x dims
// [128 w, 128 w + 128), V: keys [w kVKeys, ..) x the CTA's half of the dims, in
// the layouts that the TMA copies of shared tiles make.  Keys that do not exist
// are zeros (no weight is on them, and nothing is known of their memory).
template <int DP, bool FP8, bool V>
CSA_DEVINL void gather_slot(const Params &p, const Tile &t, int rank, int w, uint32_t dst) {
    using Lt = Layout<DP>;
    const AttendArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    constexpr int kKeys = V ? Lt::kVKeys : 64, kPer = kKeys / 32, kUnits = V ? Lt::kVChunks * 8 : 16;  // 8-dim units per key
    const int key0 = V ? w * kKeys : rank * 64, dim0 = V ? rank * (DP / 2) : w * 128;
    // rows of keys key0 + lane, + 32, ..: index, ~index in the rings, or none
    constexpr long long kNone = 0x7fffffffffffffffLL;
    long long row[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const long long k = t.first + key0 + i * 32 + lane;
        row[i] = kNone;
        if (k < t.own.n_own) {
            const uint32_t e = (uint32_t)(p.n_shared + k);
            const int id = __ldg(a.table + (size_t)t.b * a.max_pages + e / (uint32_t)a.page);
            if (id >= 0 && id < a.n_pages) row[i] = (long long)id * a.page + e % (uint32_t)a.page;
        } else if (k < t.own.total) {
            const uint32_t u = (uint32_t)(t.own.u0 + (int)(k - t.own.n_own));
            row[i] = ~((long long)t.b * a.win_rows + u % (uint32_t)a.win_rows);
        }
    }
    // shared-memory address of 16-byte unit u of key k (both within the slot)
    const auto at = [&](int k, int u) {
        const uint32_t base = V ? (uint32_t)(k / p.vbox * (Lt::kVChunks * p.vbox) + (u >> 3) * p.vbox + k % p.vbox) * 128
                                : (uint32_t)(u >> 3) * 8192 + k * 128;
        return dst + base + (((u & 7) ^ (k & 7)) << 4);
    };
    if constexpr (FP8) {
        constexpr int kU2 = kUnits / 2;  // 16 codes each
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
#pragma unroll
            for (int c0 = 0; c0 < kU2; c0 += 8) {  // 32 * kU2 units of these 32 keys, 8 loads in flight
                uint4 v[8];
                uint32_t e[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int q = (c0 + c) * 32 + lane, k = q / kU2, d = dim0 + (q % kU2) * 16;
                    const long long r = __shfl_sync(0xffffffffu, row[i], k);
                    v[c] = make_uint4(0u, 0u, 0u, 0u);
                    e[c] = 0u;
                    if (r != kNone) {
                        const size_t ri = (size_t)(r < 0 ? ~r : r);
                        v[c] = ldg16((r < 0 ? a.win8 : a.kv8) + ri * a.D + d);
                        e[c] = __ldg((r < 0 ? a.win8e : a.kv8e) + ri * (a.D / 128) + d / 128);
                    }
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int q = (c0 + c) * 32 + lane, k = i * 32 + q / kU2, u = (q % kU2) * 2;
                    const uint4 lo = e4m3x8_bf16x8(make_uint2(v[c].x, v[c].y), e[c]);
                    const uint4 hi = e4m3x8_bf16x8(make_uint2(v[c].z, v[c].w), e[c]);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(k, u)), "r"(lo.x), "r"(lo.y), "r"(lo.z),
                                 "r"(lo.w)
                                 : "memory");
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(k, u + 1)), "r"(hi.x), "r"(hi.y),
                                 "r"(hi.z), "r"(hi.w)
                                 : "memory");
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
#pragma unroll 8
            for (int c = 0; c < kUnits; ++c) {
                const int q = c * 32 + lane, k = q / kUnits, u = q % kUnits, d = dim0 + u * 8;
                const long long r = __shfl_sync(0xffffffffu, row[i], k);
                const bool there = r != kNone && d < a.D;
                const uint16_t *src = (r < 0 ? a.win + (size_t)~r * a.D : a.kv + (size_t)r * a.D) + d;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(i * 32 + k, u)),
                             "l"(there ? src : a.win), "r"(there ? 16 : 0)
                             : "memory");
            }
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
        for (int i = 0; i < kSlots; ++i) {
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
        for (int i = 0; i < kProducers; ++i) mbar_init(s.vfix + i, 1);
        *s.abort_flag = 0;
        fence_mbar_init();
        tc::prefetch_tmap(&qmap);
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
    }
    if (warp == kQueryWarp) tc::tmem_alloc_2sm(smem_u32(s.tmem_slot), 512);
    if (warp == kSoftWarp0) deal_units(p, s, pair, blockIdx.x == 0);
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();  // both CTAs' barriers exist
    tc::fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = *s.tmem_slot;

    if (warp < kProducers) {
        // ------------------------------------------------------------ producers
        // The copies of an own slot are in flight while the warp's next slot is issued (unless
        // that one is not free yet).  TMA copies are issued by one thread inside an elect_one
        // branch (one issued by every lane under a guard, or by a diverged lane, took ~200
        // cycles: more than the MMAs that it feeds).
        if (p.linear) asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows' copy
        const uint32_t full0 = tc::map_to_rank(smem_u32(s.full), 0), slots = smem_u32(s.slots);
        const uint32_t vfix = tc::map_to_rank(smem_u32(s.vfix + warp), rank);
        uint32_t it = 0, nfix = 0;
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
        // ring position `it`: slot w of a tile's K or V
        const auto fill = [&](bool v, uint32_t w, const Tile &t, const Range &rg) {
            if (!ok || (it & (kProducers - 1)) != (uint32_t)warp) return;
            const uint32_t sl = it % kSlots, par = ((it / kSlots) & 1u) ^ 1u, empty = smem_u32(s.empty + sl);
            const uint32_t dst = slots + sl * kSlotBytes;
            if (!__all_sync(0xffffffffu, mbar_test_wait(empty, par))) {
                flush();
                if (!(ok = warp_wait(empty, par, p.ctx, s.abort_flag))) return;
            }
            if (!t.shared()) {
                if (v) gather_slot<DP, FP8, true>(p, t, rank, w, dst);
                else gather_slot<DP, FP8, false>(p, t, rank, w, dst);
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
                return;
            }
            // row of 16 entries `lane` of the tile: below 0 (which reads as zeros) where no row
            // sees them or their page does not exist
            const int key = (int)t.first + lane * 16;
            int row = -kPrefixKeys;
            if (lane < 8 && key < rg.vmax) {
                if (p.linear) {
                    row = key;
                } else {
                    const int id = __ldg(a.table + (uint32_t)key / (uint32_t)a.page);
                    if (id >= 0 && id < a.n_pages) row = id * a.page + (int)((uint32_t)key % (uint32_t)a.page);
                }
            }
            if (!v) {
                const int g0 = rank * 4, r0 = __shfl_sync(0xffffffffu, row, g0), r1 = __shfl_sync(0xffffffffu, row, g0 + 1);
                const int r2 = __shfl_sync(0xffffffffu, row, g0 + 2), r3 = __shfl_sync(0xffffffffu, row, g0 + 3);
                if (tc::elect_one()) {
                    const uint32_t bar = full0 + sl * 8;
                    mbar_arrive_expect_tx_cluster(bar, kSlotBytes);
                    if (p.box == 64) {
                        tc::tma_load_3d_2sm(dst, &kmap, bar, 0, r0, 2 * w);
                    } else {
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t d = dst + c * 8192;
                            tc::tma_load_3d_2sm(d, &kmap, bar, 0, r0, 2 * w + c);
                            if (p.box == 16) tc::tma_load_3d_2sm(d + 16 * 128, &kmap, bar, 0, r1, 2 * w + c);
                            tc::tma_load_3d_2sm(d + 32 * 128, &kmap, bar, 0, r2, 2 * w + c);
                            if (p.box == 16) tc::tma_load_3d_2sm(d + 48 * 128, &kmap, bar, 0, r3, 2 * w + c);
                        }
                    }
                }
                __syncwarp();
                return;
            }
            // V: entries of the tile that do not count have zero weights; their values (anything, in
            // memory) are cleared where a copy brings them
            const int end = rg.vmax - (int)t.first - (int)w * Lt::kVKeys;  // entries of the slot that count
            const bool fix = end > 0 && end < Lt::kVKeys && end % p.vbox != 0;
            constexpr int kGroups = Lt::kVKeys / 16;
            int r[kGroups];
#pragma unroll
            for (int i = 0; i < kGroups; ++i) r[i] = __shfl_sync(0xffffffffu, row, w * kGroups + i);
            if (tc::elect_one()) {
                const uint32_t bar = fix ? vfix : full0 + sl * 8;
                mbar_arrive_expect_tx_cluster(bar, kSlotBytes);
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
                    if (i * 16 % p.vbox == 0)
                        tc::tma_load_3d_2sm(dst + i * 16 * (Lt::kVChunks * 128), &vmap, bar, 0, r[i], rank * Lt::kVChunks);
            }
            __syncwarp();
            if (fix) {
                if (!(ok = warp_wait(smem_u32(s.vfix + warp), nfix & 1u, p.ctx, s.abort_flag))) return;
                ++nfix;
                // entry e of the slot, chunk c: [e / vbox][c][e % vbox][128 B]
                uint4 *slot = reinterpret_cast<uint4 *>(s.slots + sl * kSlotBytes);
                for (int y = lane; y < Lt::kVKeys * Lt::kVChunks * 8; y += 32) {
                    const int line = y >> 3, e = line / (Lt::kVChunks * p.vbox) * p.vbox + line % p.vbox;
                    if (e >= end) slot[y] = make_uint4(0u, 0u, 0u, 0u);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                mbar_arrive_cluster(full0 + sl * 8, lane == 0);
            }
        };
        Range rg;
        for (Walk wk(s); ok && wk.next(p, rg);) {
            Tiles k(p, rg);
            Tile v = k.t;
            for (int j = 0; j <= rg.n && ok; ++j) {
                if (j < rg.n) {
                    if (j > 0) {
                        v = k.t;
                        k.next(p, rg);
                    }
                    for (uint32_t w = 0; w < Lt::kPieces; ++w, ++it) fill(false, w, k.t, rg);
                } else {
                    v = k.t;
                }
                if (j > 0)
                    for (uint32_t w = 0; w < Lt::kPieces; ++w, ++it) fill(true, w, v, rg);
            }
        }
        if (ok) flush();
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!ok) {  // given up: TMA copies may still be in flight to this shared memory
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
        }
    } else if (warp == kMmaWarp && rank == 0) {
        // ------------------------------------------------------------ MMA issuer (one thread)
        const uint64_t qdesc = tc::smem_desc(smem_u32(s.q), 1024, tc::kLayoutSw128);
        const uint64_t kdesc = tc::smem_desc(smem_u32(s.slots), 1024, tc::kLayoutSw128);
        // V as stored, [keys][dims] (MN-major): 64-dim chunks vbox * 128 bytes apart, 8-key groups 1024
        const uint64_t vdesc = tc::smem_desc_lbo(smem_u32(s.slots), p.vbox * 128, 1024, tc::kLayoutSw128);
        const uint64_t pdesc = tc::smem_desc(smem_u32(s.p), 1024, tc::kLayoutSw128);
        uint32_t it0 = 0, g0 = 0, nq = 0;
        Range rg;
        for (Walk wk(s); wk.next(p, rg);) {
            if (tc::elect_one()) {
                uint32_t it = it0;
                bool ok = mbar_wait(smem_u32(s.qready), nq & 1u, p.ctx, s.abort_flag);
                for (int j = 0; j <= rg.n && ok; ++j) {
                    if (j < rg.n) {
                        const uint32_t g = g0 + j, b = g & 1u;
                        if (!(ok = mbar_wait(smem_u32(s.sempty + b), ((g >> 1) & 1u) ^ 1u, p.ctx, s.abort_flag))) break;
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
                        if (j + 1 == rg.n) tc::mma_commit_2sm(smem_u32(s.qempty));
                    }
                    if (j > 0) {
                        const uint32_t g = g0 + j - 1, b = g & 1u;
                        if (!(ok = mbar_wait(smem_u32(s.pfull + b), (g >> 1) & 1u, p.ctx, s.abort_flag))) break;
                        for (int w = 0; w < Lt::kPieces; ++w, ++it) {
                            const uint32_t sl = it % kSlots;
                            if (!(ok = mbar_wait(smem_u32(s.full + sl), (it / kSlots) & 1u, p.ctx, s.abort_flag))) break;
                            tc::fence_after_sync();
#pragma unroll
                            for (int k = 0; k < Lt::kVKeys / 16; ++k) {  // 16 keys each
                                const uint32_t kt = w * (Lt::kVKeys / 16) + k;
                                const uint32_t x = k * 16, voff = x / p.vbox * (Lt::kVChunks * p.vbox * 128) + x % p.vbox * 128;
#pragma unroll
                                for (int i = 0; i < Lt::kPvMmas; ++i)
                                    tc::mma_f16_2sm(tmem + i * (Lt::kPvN / 2),
                                                    pdesc + ((b * kPBytes + (kt >> 2) * 8192 + (kt & 3) * 32) >> 4),
                                                    vdesc + ((sl * kSlotBytes + voff + i * 2 * p.vbox * 128) >> 4), p.idesc_pv,
                                                    (j > 1 || kt) ? 1u : 0u);
                            }
                            tc::mma_commit_2sm(smem_u32(s.empty + sl));
                        }
                        if (!ok) break;
                        tc::mma_commit_2sm(smem_u32(s.pvdone + b));
                    }
                }
            }
            __syncwarp();
            if (*(volatile int *)s.abort_flag) break;
            it0 += rg.n * 2 * Lt::kPieces;
            g0 += rg.n;
            ++nq;
        }
    } else if (warp == kQueryWarp) {
        // ------------------------------------------------------------ query tiles
        const uint32_t qland = tc::map_to_rank(smem_u32(s.qland), rank), qready0 = tc::map_to_rank(smem_u32(s.qready), 0);
        uint32_t nq = 0;
        bool ok = true;
        Range rg;
        for (Walk wk(s); wk.next(p, rg); ++nq) {
            if (!(ok = warp_wait(smem_u32(s.qempty), (nq & 1u) ^ 1u, p.ctx, s.abort_flag))) break;
            if (tc::elect_one()) {
                mbar_arrive_expect_tx_cluster(qland, Lt::kQBytes);
                for (int c = 0; c < DP / 64; c += 2)
                    tc::tma_load_3d_2sm(smem_u32(s.q) + c * 8192, &qmap, qland, 0, rg.rt * kPrefixRows + rank * 64, c);
            }
            __syncwarp();
            if (!(ok = warp_wait(smem_u32(s.qland), nq & 1u, p.ctx, s.abort_flag))) break;
            if (!q_rw) mbar_arrive_cluster(qready0, lane == 0);  // else the softmax warps rewrite the tile first
        }
        if (!ok) {  // as above
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
        }
    } else if (warp >= kSoftWarp0) {
        // ------------------------------------------------------------ softmax, partial rows
        // A wait that was given up (the abort flag makes all later ones return at once) does
        // not end a warp's loops: the four warps of 32 rows meet at named barriers.
        const int quarter = warp & 3, wg = (warp - kSoftWarp0) >> 2;
        const int tl = quarter * 32 + lane;       // tensor-memory lane
        const int r = tl & 63, hf = tl >> 6;      // row of this CTA's 64; first / second half of the columns
        const int q4 = hf * 2 + wg;               // which of the row's four threads
        const int bar_id = 1 + (quarter & 1);     // the 128 threads of 32 rows
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t sempty0 = tc::map_to_rank(smem_u32(s.sempty), 0), pfull0 = tc::map_to_rank(smem_u32(s.pfull), 0);
        const uint32_t qready0 = tc::map_to_rank(smem_u32(s.qready), 0);
        const int n_rows = (int)(a.n_bq * a.H);
        uint32_t g = 0, nq = 0;
        Range rg;
        for (Walk wk(s); wk.next(p, rg);) {
            const size_t pi = (size_t)pair + rg.rt;
            const int row = rg.rt * kPrefixRows + rank * 64 + r;
            const int bq = row < n_rows ? row / a.H : 0, b_row = bq / a.nq;
            const int t = row < n_rows ? __ldg(a.q_pos + bq) : -1;
            const int vis = visible(p, t, p.n_shared);
            // shared entries need a mask only past the fewest that a row of this warp sees, or
            // where a page is missing
            const int vis_min = __reduce_min_sync(0xffffffffu, vis);
            bool holes = false;
            if (rg.x < rg.shared)
                for (int pg = rg.x * kPrefixKeys / a.page + lane; (long long)pg * a.page < rg.vmax; pg += 32) {
                    const int id = __ldg(a.table + pg);
                    holes |= id < 0 || id >= a.n_pages;
                }
            holes = __any_sync(0xffffffffu, holes);
            warp_wait(smem_u32(s.qland), nq & 1u, p.ctx, s.abort_flag);
            ++nq;
            s.xsum[q4 * 64 + r] = query_units<DP>(a, s.q, r, q4, t, q_rw);
            if (q_rw) tc::fence_proxy_async_smem();
            __syncwarp();
            if (q_rw) mbar_arrive_cluster(qready0, lane == 0);
            mbar_arrive(smem_u32(s.qempty), lane == 0);
            group_sync(bar_id);
            const float ss = (s.xsum[r] + s.xsum[64 + r]) + (s.xsum[128 + r] + s.xsum[192 + r]);
            group_sync(bar_id);
            // 1 / RMS times the softmax scale, in log2 units
            const float rq = (1.0f / sqrtf(ss / (float)a.D + a.eps)) * a.scale * 1.4426950408889634f;

            float m_run = -INFINITY, l = 0.f;
            Tiles tile(p, rg);
            for (int j = 0; j < rg.n; ++j, ++g) {
                const uint32_t b = g & 1u, ph = (g >> 1) & 1u;
                if (j > 0) tile.next(p, rg);
                const Tile &tl_ = tile.t;
                const int off = hf * 64 + wg * 32;
                uint32_t mask = 0xffffffffu;  // which of this thread's 32 keys take part
                bool whole = tl_.shared() && !holes && (int)tl_.first + off + 32 <= vis_min;
                if (!whole) {
                    mask = key_mask(p, tl_, off, t, vis, b_row);
                    whole = __all_sync(0xffffffffu, mask == 0xffffffffu);
                }
                warp_wait(smem_u32(s.sfull + b), ph, p.ctx, s.abort_flag);
                tc::fence_after_sync();
                float sc[32];
                tc::tmem_ld32(tmem + lane_base + kSCols + b * 64 + wg * 32, sc);
                tc::tmem_wait_ld();
                tc::fence_before_sync();
                __syncwarp();
                mbar_arrive_cluster(sempty0 + b * 8, lane == 0);
#pragma unroll
                for (int i = 0; i < 32; ++i) sc[i] *= rq;
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) sc[i] = (mask >> i) & 1u ? sc[i] : -INFINITY;
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], sc[i]);
                float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                // the row's maximum over its four threads, each rounded to 16 bits towards zero
                // (any reference near the maximum serves, as long as the four agree)
                s.xmax[(b * 4 + q4) * 64 + r] = (uint16_t)(__float_as_uint(mt) >> 16);
                group_sync(bar_id);
                mt = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) mt = fmaxf(mt, __uint_as_float((uint32_t)s.xmax[(b * 4 + i) * 64 + r] << 16));
                const bool mine = m_run != -INFINITY && mt > m_run + kRescaleThreshold;
                if (__any_sync(0xffffffffu, mine)) {
                    const uint32_t gp = g - 1;  // O after the P.V of the tile before
                    warp_wait(smem_u32(s.pvdone + (gp & 1u)), (gp >> 1) & 1u, p.ctx, s.abort_flag);
                    tc::fence_after_sync();
                    const float f = mine ? exp2f(m_run - mt) : 1.0f;
                    for (int c = wg * (DP / 4); c < (wg + 1) * (DP / 4); c += 32) {
                        float v[32];
                        tc::tmem_ld32(tmem + lane_base + c, v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= f;
                        tc::tmem_st32(tmem + lane_base + c, v);
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
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float p0 = exp2_ftz(sc[i] - mref), p1 = exp2_ftz(sc[i + 1] - mref);
                    ps[0] += p0;
                    ps[1] += p1;
                    pk[i / 2] = pack_bf16x2(p0, p1);
                }
                l += ps[0] + ps[1];
                // P buffer b was read by the P.V of tile g - 2
                warp_wait(smem_u32(s.pvdone + b), ph ^ 1u, p.ctx, s.abort_flag);
                uint8_t *prow = s.p + b * kPBytes + hf * 8192 + r * 128;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    *reinterpret_cast<uint4 *>(prow + (((wg * 4 + x) ^ (r & 7)) << 4)) =
                        make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
                tc::fence_proxy_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                mbar_arrive_cluster(pfull0 + b * 8, lane == 0);
            }
            const uint32_t gl = g - 1;
            warp_wait(smem_u32(s.pvdone + (gl & 1u)), (gl >> 1) & 1u, p.ctx, s.abort_flag);
            tc::fence_after_sync();
            s.xsum[q4 * 64 + r] = l;  // every thread is past its last tile's maxima
            group_sync(bar_id);
            if (q4 == 0)
                p.ml[pi * kPrefixRows + rank * 64 + r] =
                    make_float2(m_run, (s.xsum[r] + s.xsum[64 + r]) + (s.xsum[128 + r] + s.xsum[192 + r]));
            group_sync(bar_id);
            float4 *dst = reinterpret_cast<float4 *>(p.part) + (pi * 2 + rank) * (DP / 8) * 128 + tl;
            for (int c = wg * (DP / 4); c < (wg + 1) * (DP / 4); c += 32) {
                float v[32];
                tc::tmem_ld32(tmem + lane_base + c, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dst[(size_t)(c / 4 + i) * 128] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
            tc::fence_before_sync();  // O is read before the next range's first P.V (through pfull)
        }
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
