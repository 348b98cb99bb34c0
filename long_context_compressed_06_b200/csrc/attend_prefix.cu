// attend_prefix.cu -- attention of a whole batch over the entries that all its
// requests share, as one product (the n_shared part of hca_attend_paged).
//
// With the query rows of every request stacked, Q is [R = batch * nq * H][D]
// and the shared entries X [n_shared][D] are keys and values of all of them:
//   S = scale / RMS(q) * Q X^T,   P = exp2(S - m),   O = P X
// with the running maximum m and sum l of every row kept per tile of 128
// entries (m raised only when it grows by more than 2^8, so that O in tensor
// memory is rarely rescaled).  O, m and l of a tile range go out in 32 bits and
// are merged with each request's own entries and window.
//
// A pair of SMs owns 128 rows (cta_group::2, M = 128): every MMA reads half of
// its B operand from each SM, and an accumulator takes 64 rows x N/2 columns x
// two lane halves of each SM's tensor memory, so that O at D = 512 fits in 256
// columns beside two S buffers.  One SM alone would have to run at M = 64, half
// the tensor rate (128 rows x 512 fp32 columns fill its tensor memory).
// Column c of lane half f of O is dim f * DP / 2 + c.
// The price is that each SM loads 64 of a tile's 128 entries whole (its half of
// K's rows) and all 128 entries by half their dims (its half of V's columns):
// 128 KiB per SM and tile at D = 512, 1.33 times what one copy would be.
// The tensor cores' operand reads (224 KiB), these loads and P share the
// 128 B/cycle of shared memory, which bounds the kernel at D = 512.
//
// Warps: 0 TMA producer, 1 MMA issuer (the pair's leader), 2 tensor memory and
// the query tile's hand-over, 4..11 softmax (four threads per row: lane half x
// 32-column half).  16 KiB slots form one ring for both operands, in the order
// the MMAs consume them (K0, K1, V0, K2, V1, ...).  Work: see PrefixPlan.
#include <algorithm>
#include <cstring>

#include "attend_common.cuh"
#include "common.cuh"
#include "kernels.h"
#include "quant_fp8.cuh"
#include "tc.cuh"

namespace csa {
namespace {

constexpr int kThreads = 384;
constexpr int kSoftWarp0 = 4, kSoftWarps = 8;
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
    int *rows;       // [2][8] first rows of a tile's key groups (producer)
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
    s.rows = reinterpret_cast<int *>(s.vfix + 1);
    s.tmem_slot = reinterpret_cast<uint32_t *>(s.rows + 16);
    s.abort_flag = reinterpret_cast<int *>(s.tmem_slot + 1);
    return s;
}

template <int DP>
constexpr size_t smem_bytes() {
    return 1024 + Layout<DP>::kQBytes + kSlots * kSlotBytes + 2 * kPBytes + 1024 + (2 * kSlots + 12) * 8 + 64 + 16;
}
static_assert(smem_bytes<512>() <= 227 * 1024, "shared memory of one CTA");

// A pair's part of one row tile: tiles [k0, k0 + n) of 128 entries, vmax the
// most entries that any row of the tile sees.  Tiles past vmax are left out.
struct Range {
    int rt, k0, n, vmax;
    long long next;  // first unit after the range
};

// warp-collective
CSA_DEVINL Range range_at(const Params &p, long long u, long long u1) {
    Range r;
    const int KT = p.plan.key_tiles;
    r.rt = (int)(u / KT);
    r.k0 = (int)(u - (long long)r.rt * KT);
    const int k1 = (int)std::min<long long>(KT, r.k0 + (u1 - u));
    r.next = u + (k1 - r.k0);
    const long long row0 = (long long)r.rt * kPrefixRows;
    const long long b0 = row0 / p.a.H, b1 = std::min(p.a.n_bq - 1, (row0 + kPrefixRows - 1) / p.a.H);
    int v = 0;
    for (long long b = b0 + (threadIdx.x & 31); b <= b1; b += 32)
        v = std::max(v, (int)n_visible(__ldg(p.a.q_pos + b), p.a.m, p.n_shared));
    r.vmax = __reduce_max_sync(0xffffffffu, v);
    r.n = std::max(0, std::min(k1, (r.vmax + kPrefixKeys - 1) / kPrefixKeys) - r.k0);
    return r;
}

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

template <int DP>
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
        mbar_init(s.vfix, 1);
        *s.abort_flag = 0;
        fence_mbar_init();
        tc::prefetch_tmap(&qmap);
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
    }
    if (warp == 2) tc::tmem_alloc_2sm(smem_u32(s.tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();  // both CTAs' barriers exist
    tc::fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = *s.tmem_slot;
    const long long u0 = p.plan.first(pair), u1 = p.plan.first(pair + 1);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        // One thread issues, inside an elect_one branch (a copy issued by every lane under a
        // guard, or a diverged lane, took ~200 cycles each: more than the MMAs that it feeds).
        if (p.linear) asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows' copy
        const uint32_t full0 = tc::map_to_rank(smem_u32(s.full), 0), slots = smem_u32(s.slots);
        const uint32_t qland = tc::map_to_rank(smem_u32(s.qland), rank), vfix = tc::map_to_rank(smem_u32(s.vfix), rank);
        uint32_t it0 = 0, nq = 0, nfix = 0;
        bool ok = true;
        for (long long u = u0; u < u1 && ok;) {
            const Range rg = range_at(p, u, u1);
            u = rg.next;
            if (rg.n == 0) continue;
            if (!(ok = warp_wait(smem_u32(s.qempty), (nq & 1u) ^ 1u, p.ctx, s.abort_flag))) break;
            ++nq;
            if (tc::elect_one()) {
                mbar_arrive_expect_tx_cluster(qland, Lt::kQBytes);
                for (int c = 0; c < DP / 64; c += 2)
                    tc::tma_load_3d_2sm(smem_u32(s.q) + c * 8192, &qmap, qland, 0, rg.rt * kPrefixRows + rank * 64, c);
            }
            // row of 16 entries `lane` of tile j: below 0 (which reads as zeros) where no row
            // sees them or their page does not exist
            const auto tile_rows = [&](int j) {
                const int key = (rg.k0 + j) * kPrefixKeys + lane * 16;
                if (lane < 8) {
                    int row = -kPrefixKeys;
                    if (key < rg.vmax) {
                        if (p.linear) {
                            row = key;
                        } else {
                            const int id = __ldg(a.table + (uint32_t)key / (uint32_t)a.page);
                            if (id >= 0 && id < a.n_pages) row = id * a.page + (int)((uint32_t)key % (uint32_t)a.page);
                        }
                    }
                    s.rows[(j & 1) * 8 + lane] = row;
                }
                __syncwarp();
            };
            tile_rows(0);
            for (int j = 0; j <= rg.n && ok; ++j) {
                // entries of V's tile that count; the others' weights are zero, their values
                // (anything, in memory) are cleared where a copy brings them
                const int end = rg.vmax - (rg.k0 + j - 1) * kPrefixKeys;
                const bool fix = j > 0 && end < kPrefixKeys && end % p.vbox != 0;
                bool good = true;
                if (tc::elect_one()) {
                    uint32_t it = it0;
                    if (j < rg.n) {
                        const int *rows = s.rows + (j & 1) * 8 + rank * 4;
                        for (int w = 0; w < Lt::kPieces && good; ++w, ++it) {
                            const uint32_t sl = it % kSlots, dst = slots + sl * kSlotBytes, bar = full0 + sl * 8;
                            if (!(good = mbar_wait(smem_u32(s.empty + sl), ((it / kSlots) & 1u) ^ 1u, p.ctx, s.abort_flag)))
                                break;
                            mbar_arrive_expect_tx_cluster(bar, kSlotBytes);
                            if (p.box == 64) {
                                tc::tma_load_3d_2sm(dst, &kmap, bar, 0, rows[0], 2 * w);
                            } else {
                                for (int x = 0; x < 64; x += p.box) {
                                    const int row = rows[x / 16];
                                    tc::tma_load_3d_2sm(dst + x * 128, &kmap, bar, 0, row, 2 * w);
                                    tc::tma_load_3d_2sm(dst + 8192 + x * 128, &kmap, bar, 0, row, 2 * w + 1);
                                }
                            }
                        }
                    }
                    if (j > 0 && !fix) {
                        const int *rows = s.rows + ((j - 1) & 1) * 8;
                        for (int w = 0; w < Lt::kPieces && good; ++w, ++it) {
                            const uint32_t sl = it % kSlots, dst = slots + sl * kSlotBytes, bar = full0 + sl * 8;
                            if (!(good = mbar_wait(smem_u32(s.empty + sl), ((it / kSlots) & 1u) ^ 1u, p.ctx, s.abort_flag)))
                                break;
                            mbar_arrive_expect_tx_cluster(bar, kSlotBytes);
                            for (int x = 0; x < Lt::kVKeys; x += p.vbox)
                                tc::tma_load_3d_2sm(dst + x * (Lt::kVChunks * 128), &vmap, bar, 0,
                                                    rows[(w * Lt::kVKeys + x) / 16], rank * Lt::kVChunks);
                        }
                    }
                }
                __syncwarp();
                ok = good && !*(volatile int *)s.abort_flag;
                ok = __all_sync(0xffffffffu, ok);
                it0 += j < rg.n ? Lt::kPieces : 0;
                if (fix) {
                    const int *rows = s.rows + ((j - 1) & 1) * 8;
                    for (int w = 0; w < Lt::kPieces && ok; ++w) {
                        const uint32_t it = it0 + w, sl = it % kSlots, dst = slots + sl * kSlotBytes;
                        if (!(ok = warp_wait(smem_u32(s.empty + sl), ((it / kSlots) & 1u) ^ 1u, p.ctx, s.abort_flag))) break;
                        if (tc::elect_one()) {
                            mbar_arrive_expect_tx_cluster(vfix, kSlotBytes);
                            for (int x = 0; x < Lt::kVKeys; x += p.vbox)
                                tc::tma_load_3d_2sm(dst + x * (Lt::kVChunks * 128), &vmap, vfix, 0,
                                                    rows[(w * Lt::kVKeys + x) / 16], rank * Lt::kVChunks);
                        }
                        __syncwarp();
                        if (!(ok = warp_wait(smem_u32(s.vfix), nfix & 1u, p.ctx, s.abort_flag))) break;
                        ++nfix;
                        // entry e of the slot, chunk c: [e / vbox][c][e % vbox][128 B]
                        uint8_t *slot = s.slots + sl * kSlotBytes;
                        for (int x = lane; x < (Lt::kVKeys * Lt::kVChunks) * 8; x += 32) {
                            const int row = x >> 3, e = row / (Lt::kVChunks * p.vbox) * p.vbox + row % p.vbox;
                            if (w * Lt::kVKeys + e >= end) reinterpret_cast<uint4 *>(slot)[x] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        mbar_arrive_cluster(full0 + sl * 8, lane == 0);
                    }
                }
                it0 += j > 0 ? Lt::kPieces : 0;
                if (j + 1 < rg.n) tile_rows(j + 1);
            }
        }
        if (!ok) {  // given up: copies may still be in flight to this shared memory
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
        }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ MMA issuer (one thread)
        const uint64_t qdesc = tc::smem_desc(smem_u32(s.q), 1024, tc::kLayoutSw128);
        const uint64_t kdesc = tc::smem_desc(smem_u32(s.slots), 1024, tc::kLayoutSw128);
        // V as stored, [keys][dims] (MN-major): 64-dim chunks vbox * 128 bytes apart, 8-key groups 1024
        const uint64_t vdesc = tc::smem_desc_lbo(smem_u32(s.slots), p.vbox * 128, 1024, tc::kLayoutSw128);
        const uint64_t pdesc = tc::smem_desc(smem_u32(s.p), 1024, tc::kLayoutSw128);
        uint32_t it0 = 0, g0 = 0, nq = 0;
        for (long long u = u0; u < u1;) {
            const Range rg = range_at(p, u, u1);
            u = rg.next;
            if (rg.n == 0) continue;
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
    } else if (warp == 2) {
        // ------------------------------------------------------------ query tile -> MMA issuer
        if (!q_rw) {
            const uint32_t qready0 = tc::map_to_rank(smem_u32(s.qready), 0);
            uint32_t nq = 0;
            for (long long u = u0; u < u1;) {
                const Range rg = range_at(p, u, u1);
                u = rg.next;
                if (rg.n == 0) continue;
                if (!warp_wait(smem_u32(s.qland), nq & 1u, p.ctx, s.abort_flag)) break;
                mbar_arrive_cluster(qready0, lane == 0);
                ++nq;
            }
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
        const long long n_rows = a.n_bq * a.H;
        uint32_t g = 0, nq = 0;
        for (long long u = u0; u < u1;) {
            const Range rg = range_at(p, u, u1);
            u = rg.next;
            const size_t pi = (size_t)pair + rg.rt;
            if (rg.n == 0) {
                if (q4 == 0) p.ml[pi * kPrefixRows + rank * 64 + r] = make_float2(-INFINITY, 0.f);
                continue;
            }
            const long long row = (long long)rg.rt * kPrefixRows + rank * 64 + r;
            const long long t = row < n_rows ? __ldg(a.q_pos + row / a.H) : -1;
            const int vis = (int)n_visible(t, a.m, p.n_shared);
            // entries of a tile need a mask only past the fewest that a row of this warp sees,
            // or where a page is missing
            const int vis_min = __reduce_min_sync(0xffffffffu, vis);
            bool holes = false;
            for (int pg = rg.k0 * kPrefixKeys / a.page + lane; (long long)pg * a.page < rg.vmax; pg += 32) {
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
            for (int j = 0; j < rg.n; ++j, ++g) {
                const uint32_t b = g & 1u, ph = (g >> 1) & 1u;
                const int key = (rg.k0 + j) * kPrefixKeys + hf * 64 + wg * 32;
                const bool whole = !holes && key + 32 <= vis_min;
                uint32_t mask = 0xffffffffu;  // which of this thread's 32 entries take part
                if (!whole) {
                    const int lim = vis - key;
                    mask = lim >= 32 ? 0xffffffffu : (lim <= 0 ? 0u : (1u << lim) - 1u);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (lim > 16 * h) {
                            const int id = __ldg(a.table + (uint32_t)(key + 16 * h) / (uint32_t)a.page);
                            if (id < 0 || id >= a.n_pages) mask &= h ? 0x0000ffffu : 0xffff0000u;
                        }
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
            float4 *dst = reinterpret_cast<float4 *>(p.part) + ((pi * 2 + rank) * (DP / 16) * 128 + tl) * 2;
            for (int c = wg * (DP / 4); c < (wg + 1) * (DP / 4); c += 32) {
                float v[32];
                tc::tmem_ld32(tmem + lane_base + c, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dst[(size_t)(c / 8 + i / 2) * 256 + (i & 1)] =
                        make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
            tc::fence_before_sync();  // O is read before the next range's first P.V (through pfull)
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();  // no arrival of the other CTA is outstanding
    if (warp == 2) {
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

template <int DP>
int launch_d(const PrefixArgs &x, const DevCtx &ctx, cudaStream_t st) {
    Params p = {};
    p.a = x.a;
    p.plan = x.plan;
    p.n_shared = (int)x.n_shared;
    p.linear = x.linear ? 1 : 0;
    p.part = x.part;
    p.ml = x.ml;
    p.ctx = ctx;
    p.idesc_qk = idesc(kPrefixKeys, false);
    p.idesc_pv = idesc(Layout<DP>::kPvN, true);
    p.box = x.linear || x.a.page % 64 == 0 ? 64 : (x.a.page % 32 == 0 ? 32 : 16);
    p.vbox = std::min(p.box, Layout<DP>::kVKeys);
    auto kern = attend_prefix_kernel<DP>;
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

PrefixPlan prefix_plan(long long rows, long long n_shared) {
    PrefixPlan pl;
    pl.row_tiles = (int)((rows + kPrefixRows - 1) / kPrefixRows);
    pl.key_tiles = (int)((n_shared + kPrefixKeys - 1) / kPrefixKeys);
    pl.pairs = (int)std::min<long long>(std::max(num_sms() / 2, 1), pl.units());
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
    switch (prefix_dims(p.a.D)) {
        case 128: return launch_d<128>(p, ctx, st);
        case 256: return launch_d<256>(p, ctx, st);
        case 512: return launch_d<512>(p, ctx, st);
        default: return CSA_ERR_UNSUPPORTED;
    }
}

}  // namespace csa
