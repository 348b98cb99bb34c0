// paged.cu -- the bookkeeping of a paged cache of compressed entries:
// csa_plan_pages (block tables and slot maps from the requests' lengths) and
// csa_paged_write / csa_paged_write_fp8kv (rows stored through a slot map).
//
// csa_plan_pages.  With e0 = old / m, e1 = (old + new) / m entries before and
// after the step, request b holds ceil(e0 / page) pages and takes the next
// ceil(e1 / page) - ceil(e0 / page) ids of the free list, requests in order; three
// prefix sums over the batch (tokens, entries, pages) place everything else.
// The kernel is bound by latency (a decode step) or by the 8 bytes per entry
// and 12 per token that it writes (a prompt).
//
// Up to kFusedBatch requests one launch does it all: every block forms the
// three prefix sums over the whole batch in its shared memory (the lengths are
// 8 bytes a request, read from L2; the sums saturate at 2^32 - 1 there, past
// every place that is filled) and fills its own range of the outputs.  Above
// that a one-block launch writes the sums to global memory first and the filling
// blocks search them there.  5000 requests of up to 3 tokens each take 10 us
// (27 us in two launches: 14 for one block's sums, the rest mostly the
// thirteen dependent loads from L2 of every search).  The blocks' own sums grow
// with the batch: 16384 requests take 67 us, where 16385, in two launches, take 49;
// the limit stands where the sums still fit and no workspace is asked for.  100000
// requests take 291 us and 2^20 2.9 ms, nearly all of it the one block's scan.
#include "common.cuh"
#include "kernels.h"
#include "quant_fp8.cuh"
#include "tc.cuh"

namespace csa {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kFusedBatch = 16384;  // three 32-bit sums per request: 192 KiB of shared memory
constexpr int kPlanItems = 1024;    // outputs per filling block

struct Plan : PlanArgs {
    FastDiv fm, fpage, fring;  // m, page, ring
};

struct Req {
    int o, n, e0, e1, held, fresh, cut;  // tokens, entries, pages before, pages taken, pages without a column
};

CSA_DEVINL Req request(const Plan &a, int b) {
    Req r;
    r.o = __ldg(a.old_len + b);
    r.n = __ldg(a.new_len + b);
    if (r.o < 0 || r.n < 0 || (long long)r.o + r.n > 0x7fffffffLL) r.o = r.n = 0;  // an empty slot of the batch
    r.e0 = a.fm.div(r.o);
    r.e1 = a.fm.div(r.o + r.n);
    const int h0 = a.fpage.div(r.e0), p0 = a.fpage.div(r.e1);  // ceil, without passing 31 bits
    const int h = h0 + (r.e0 - h0 * a.page ? 1 : 0), p = p0 + (r.e1 - p0 * a.page ? 1 : 0);
    r.held = min(h, a.max_pages);
    r.fresh = min(p, a.max_pages) - r.held;
    r.cut = p - h - r.fresh;
    return r;
}

struct Sums {
    long long t, e, p, cut;
};

CSA_DEVINL Sums operator+(const Sums &x, const Sums &y) { return {x.t + y.t, x.e + y.e, x.p + y.p, x.cut + y.cut}; }

CSA_DEVINL Sums shfl_up(const Sums &v, int d) {
    return {__shfl_up_sync(0xffffffffu, v.t, d), __shfl_up_sync(0xffffffffu, v.e, d),
            __shfl_up_sync(0xffffffffu, v.p, d), __shfl_up_sync(0xffffffffu, v.cut, d)};
}

struct Nothing {};  // a sum that is not kept
CSA_DEVINL void put_sum(Nothing *, long long) {}
CSA_DEVINL void put_sum(long long *at, long long v) { *at = v; }
CSA_DEVINL void put_sum(uint32_t *at, long long v) { *at = v < 0xffffffffLL ? (uint32_t)v : 0xffffffffu; }

// Exclusive prefix sums over the batch into cu_* ([batch + 1] each), by one
// block; every thread returns the totals.  A thread owns consecutive requests.
template <typename T, typename P>
CSA_DEVINL Sums scan_batch(const Plan &a, T *cu_t, T *cu_e, P *cu_p) {
    __shared__ Sums warp_tot[kPlanThreads / 32];
    const int per = (a.batch + kPlanThreads - 1) / kPlanThreads;
    const int b0 = (int)min((long long)threadIdx.x * per, (long long)a.batch), b1 = min(b0 + per, a.batch);
    Sums mine = {0, 0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        const Req r = request(a, b);
        mine = mine + Sums{r.n, r.e1 - r.e0, r.fresh, r.cut};
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums up = shfl_up(inc, d);
        if (lane >= d) inc = inc + up;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    Sums base = {0, 0, 0, 0}, total = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) base = total;
        total = total + warp_tot[w];
    }
    Sums at = {base.t + inc.t - mine.t, base.e + inc.e - mine.e, base.p + inc.p - mine.p, 0};
    for (int b = b0; b < b1; ++b) {
        const Req r = request(a, b);
        put_sum(cu_t + b, at.t);
        put_sum(cu_e + b, at.e);
        put_sum(cu_p + b, at.p);
        at = at + Sums{r.n, r.e1 - r.e0, r.fresh, 0};
    }
    if (threadIdx.x == 0) {
        put_sum(cu_t + a.batch, total.t);
        put_sum(cu_e + a.batch, total.e);
        put_sum(cu_p + a.batch, total.p);
    }
    return total;
}

CSA_DEVINL void write_counts(const Plan &a, const Sums &total) {
    const long long lacking = total.p > a.n_free ? total.p - a.n_free : 0;
    a.counts[0] = total.t;
    a.counts[1] = total.e;
    a.counts[2] = total.p;
    a.counts[3] = total.cut + lacking;
}

// the request whose range of the prefix sums holds item i < cu[batch]
template <typename T>
CSA_DEVINL int owner(const T *cu, int batch, long long i) {
    int lo = 0, hi = batch;  // cu[lo] <= i < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((long long)cu[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Fills one range of kPlanItems outputs: blocks [0, entry_blocks) the entry
// slots (and the table's new columns, by the thread of a page's first new
// entry), the others the token outputs.
template <typename T>
CSA_DEVINL void fill(const Plan &a, int block, int entry_blocks, const T *cu_t, const T *cu_e, const T *cu_p) {
    if (block < entry_blocks) {
        const long long total = cu_e[a.batch];
        // every entry of the batch has its page noted, also those past the slot map's room
        const long long all = total > a.max_entries ? total : a.max_entries;
        for (long long s = (long long)block * kPlanItems; s < all; s += (long long)entry_blocks * kPlanItems) {
            for (int k = threadIdx.x; k < kPlanItems; k += kPlanThreads) {
                const long long i = s + k;
                if (i >= all) break;
                long long slot = -1;
                if (i < total) {
                    const int b = owner(cu_e, a.batch, i);
                    const Req r = request(a, b);
                    const long long c0 = cu_e[b];
                    const int e = r.e0 + (int)(i - c0), j = a.fpage.div(e), off = e - j * a.page;
                    if (j < a.max_pages) {
                        int *cell = a.table + (size_t)b * a.max_pages + j;
                        int id;
                        if (j < r.held) {
                            id = *cell;
                        } else {
                            const long long f = cu_p[b] + (j - r.held);
                            id = f < a.n_free ? __ldg(a.free_pages + f) : -1;
                            if (off == 0) *cell = id;
                        }
                        if (id >= 0) slot = (long long)id * a.page + off;
                    }
                }
                if (i < a.max_entries) a.entry_slots[i] = slot;
            }
        }
        return;
    }
    const long long total = cu_t[a.batch], s = (long long)(block - entry_blocks) * kPlanItems;
    for (int k = threadIdx.x; k < kPlanItems; k += kPlanThreads) {
        const long long i = s + k;
        if (i >= a.max_tokens) return;
        int pos = -1;
        long long slot = -1;
        if (i < total) {
            const int b = owner(cu_t, a.batch, i);
            const int p = __ldg(a.old_len + b) + (int)(i - (long long)cu_t[b]);
            pos = p;
            // of tokens that share a ring row only the newest is kept
            if (p >= (long long)__ldg(a.old_len + b) + __ldg(a.new_len + b) - a.ring)
                slot = (long long)b * a.ring + a.fring.mod(p);
        }
        a.tok_pos[i] = pos;
        a.win_slots[i] = slot;
    }
}

__global__ void __launch_bounds__(kPlanThreads) plan_fused_kernel(const Plan a, int entry_blocks) {
    extern __shared__ uint32_t cu[];
    uint32_t *cu_t = cu, *cu_e = cu + (a.batch + 1), *cu_p = cu + 2 * (a.batch + 1);
    // the last block also writes the sums, in full
    if (blockIdx.x == gridDim.x - 1) {
        const Sums total = scan_batch(a, a.cu_tokens, a.cu_entries, (Nothing *)nullptr);
        if (threadIdx.x == 0) write_counts(a, total);
        return;
    }
    scan_batch(a, cu_t, cu_e, cu_p);
    __syncthreads();
    fill(a, blockIdx.x, entry_blocks, cu_t, cu_e, cu_p);
}

__global__ void __launch_bounds__(kPlanThreads) plan_scan_kernel(const Plan a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Sums total = scan_batch(a, a.cu_tokens, a.cu_entries, a.cu_pages);
    if (threadIdx.x == 0) write_counts(a, total);
}

__global__ void __launch_bounds__(kPlanThreads) plan_fill_kernel(const Plan a, int entry_blocks) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the sums of plan_scan_kernel
    fill(a, blockIdx.x, entry_blocks, a.cu_tokens, a.cu_entries, a.cu_pages);
}

// ---------------------------------------------------------------- writes
constexpr int kWriteThreads = 256;
// 16-byte units per thread, all in flight before the first store: 2 (13.0 us for 32770 FP8 rows of
// 512; 4: 14.3, 8: 16.6; one decode step's 256 rows 1.8, 2.5 and 4.1 us).  Slots in order or at random make no
// difference (12.8 and 12.6 us; the same rows as bf16, with a third more bytes, 8.7 and 9.0).
constexpr int kWriteUnits = 2;

// A thread's units (8 elements each) of the packed rows, and where in the pool they go (-1: nowhere):
// unit u of the rows is unit u % upr of row slots[u / upr].
struct WriteUnits {
    uint4 v[kWriteUnits];
    long long dst[kWriteUnits];
    CSA_DEVINL WriteUnits(const uint4 *__restrict__ rows, const FastDiv &upr, int units, const long long *__restrict__ slots,
                          long long n_slots) {
        const int u0 = (int)blockIdx.x * (kWriteThreads * kWriteUnits) + (int)threadIdx.x;
#pragma unroll
        for (int k = 0; k < kWriteUnits; ++k) {
            const int u = u0 + k * kWriteThreads;
            dst[k] = -1;
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (u < units) {
                v[k] = ldg_stream(rows + u);
                const int row = upr.div(u);
                const long long s = __ldg(slots + row);
                if (s >= 0 && s < n_slots) dst[k] = s * upr.d + (u - row * (int)upr.d);
            }
        }
    }
};

__global__ void __launch_bounds__(kWriteThreads)
    paged_write_kernel(const uint4 *__restrict__ rows, const FastDiv upr, int units, const long long *__restrict__ slots,
                       long long n_slots, uint4 *__restrict__ pool) {
    const WriteUnits w(rows, upr, units, slots, n_slots);
#pragma unroll
    for (int k = 0; k < kWriteUnits; ++k)
        if (w.dst[k] >= 0) pool[w.dst[k]] = w.v[k];
}

// The same with the rows quantised on the way (csa_quantize_fp8_kv's codes and
// exponents): the 16 units of a 128-channel block are 16 consecutive lanes.
__global__ void __launch_bounds__(kWriteThreads)
    paged_write_fp8_kernel(const uint4 *__restrict__ rows, const FastDiv upr, int units, const long long *__restrict__ slots,
                           long long n_slots, uint2 *__restrict__ codes, uint8_t *__restrict__ exps) {
    const WriteUnits w(rows, upr, units, slots, n_slots);
#pragma unroll
    for (int k = 0; k < kWriteUnits; ++k) {
        float f[8];
        unpack8(w.v[k], f);
        int e;
        const uint2 q = quantize_fp8_unit(f, e);  // every lane (shuffles)
        if (w.dst[k] >= 0) {
            codes[w.dst[k]] = q;
            if ((w.dst[k] & 15) == 0) exps[w.dst[k] >> 4] = (uint8_t)(e + 127);
        }
    }
}

}  // namespace

size_t plan_workspace_bytes(int batch) {
    return batch > kFusedBatch ? (size_t)(batch + 1) * sizeof(long long) : 0;
}

int launch_plan_pages(const PlanArgs &args, void *ws, cudaStream_t st) {
    Plan a;
    static_cast<PlanArgs &>(a) = args;
    const long long eb = (a.max_entries + kPlanItems - 1) / kPlanItems;
    const long long tb = (a.max_tokens + kPlanItems - 1) / kPlanItems;
    // one entry block at least: the new columns are noted also without a slot map
    const int entry_blocks = (int)(eb < 1 ? 1 : eb);
    const unsigned blocks = (unsigned)(entry_blocks + tb);
    a.fm = FastDiv::by((uint32_t)a.m);
    a.fpage = FastDiv::by((uint32_t)a.page);
    a.fring = FastDiv::by((uint32_t)a.ring);
    if (a.batch <= kFusedBatch) {
        const size_t smem = 3 * (size_t)(a.batch + 1) * sizeof(uint32_t);
        static SmemSet smem_set;
        if (!smem_set((const void *)plan_fused_kernel, 3 * (kFusedBatch + 1) * sizeof(uint32_t))) return CSA_ERR_CUDA;
        plan_fused_kernel<<<blocks + 1, kPlanThreads, smem, st>>>(a, entry_blocks);
        return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
    }
    a.cu_pages = static_cast<long long *>(ws);
    plan_scan_kernel<<<1, kPlanThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return CSA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, plan_fill_kernel, a, entry_blocks) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

int launch_paged_write(const uint16_t *rows, const long long *slots, long long n, int d, uint16_t *pool, uint8_t *codes,
                       uint8_t *exps, long long n_slots, cudaStream_t st) {
    const FastDiv upr = FastDiv::by((uint32_t)(d / 8));
    const long long most = (1LL << 30) / (d / 8);  // rows per launch: units in 31 bits
    for (long long r0 = 0; r0 < n; r0 += most) {
        const int units = (int)((n - r0 < most ? n - r0 : most) * (d / 8));
        const unsigned blocks = (unsigned)(units + kWriteThreads * kWriteUnits - 1) / (kWriteThreads * kWriteUnits);
        const uint4 *src = reinterpret_cast<const uint4 *>(rows + r0 * d);
        if (codes)
            paged_write_fp8_kernel<<<blocks, kWriteThreads, 0, st>>>(src, upr, units, slots + r0, n_slots,
                                                                     reinterpret_cast<uint2 *>(codes), exps);
        else
            paged_write_kernel<<<blocks, kWriteThreads, 0, st>>>(src, upr, units, slots + r0, n_slots,
                                                                 reinterpret_cast<uint4 *>(pool));
        if (cudaGetLastError() != cudaSuccess) return CSA_ERR_CUDA;
    }
    return CSA_OK;
}

}  // namespace csa
