// attend_common.cuh -- argument block and split-KV workspace layout shared by
// the attention kernel and the split combine.
#pragma once

#include "common.cuh"

namespace csa {

// Partial RoPE: the trailing kRopeDim channels of every head rotate in the
// rotate-half form (channel n+i with n+kRopeDim/2+i, n = D - kRopeDim): the
// normalised query at its position before the dot products, the output by the
// conjugate rotation at the same position; keys arrive already rotated.
constexpr int kRopeDim = 64;

struct AttendArgs {
    const uint16_t *q;      // [n_bq][H][D]
    const float *q_gain;    // [D] or null
    const float *sinks;     // [H] per-head sink logits (natural units) or null
    const float *rope_cos;  // [rope_npos][kRopeDim / 2] partial-RoPE tables, or null (no RoPE)
    const float *rope_sin;  // [rope_npos][kRopeDim / 2]
    long long rope_npos;
    const uint16_t *kv;     // [batch][N][D]
    // FP8 KV cache (instead of kv / win when kv8 is set): e4m3 codes and one
    // UE8M0 exponent byte per 128 channels, value = code * 2^(e - 127)
    const uint8_t *kv8, *kv8e;    // [batch][N][D], [batch][N][D/128]
    const uint8_t *win8, *win8e;  // [batch][win_rows][D], [batch][win_rows][D/128]
    long long N;
    int m;                  // compression ratio (dense key set only)
    const int *idx;         // [n_bq][k] selected entries (CSA); unused when dense
    int k;
    bool dense;             // HCA: every visible entry is a key
    const uint16_t *win;    // [batch][win_rows][D] stream-A rows of positions win_pos0..
    long long win_pos0, win_rows;
    int W;
    // Paged cache (table set; kv / kv8 then hold [n_pages][page] rows): entry j of
    // sequence b is row table[b][j / page] * page + j % page, the window is a ring
    // of win_rows rows per sequence (position u at row u % win_rows)
    const int *table;       // [batch][max_pages] or null
    int max_pages, page;
    long long n_pages;
    const int *q_pos;       // [n_bq]
    int nq;
    long long n_bq;         // batch * nq
    int H, D;
    float scale, eps;
    uint16_t *out;          // [n_bq][H][D]
    uint16_t *part_o;       // [splits][n_bq][H][D] bf16 partial outputs, each divided by its own sum
    int part_perm;          // part_o rows of one (split, query) in warp-store order (see attend_combine)
    float2 *part_ml;        // [splits][n_bq][H] (running max in log2 units, sum)
    float *part_f;          // paged: [splits][n_bq][H][D] fp32 partial outputs, not divided, part_perm as
                            // for part_o (null: the one split's output rows are final)
    int splits;
};

// (cos, sin) of rotated pair i (< kRopeDim / 2) at position t; (1, 0) -- no
// rotation -- when RoPE is off or t lies outside the tables.
CSA_DEVINL float2 rope_cs(const AttendArgs &a, long long t, int i) {
    if (!a.rope_cos || t < 0 || t >= a.rope_npos) return make_float2(1.f, 0.f);
    const size_t o = (size_t)t * (kRopeDim / 2) + i;
    return make_float2(__ldg(a.rope_cos + o), __ldg(a.rope_sin + o));
}

int launch_attend_combine(const AttendArgs &a, cudaStream_t st);

// (running max, sum) of a paged partial row as the merge takes them; l is kTaken at least, far below any weight, in a
// row that has keys there.  A maximum of -inf is a row without keys, but neither a NaN score, which is in the sum, nor one of
// -inf raises a maximum.  Under +inf the merged row is NaN; under the lowest number the partial weighs 0 beside
// others (and 0 x inf is in its O), and alone has 0 / 0.
constexpr float kTaken = 1e-37f, kLowest = -3.402823466e38f;
CSA_DEVINL float2 partial_ml(float m, float l) {
    if (l != l) return make_float2(INFINITY, l);
    return m == -INFINITY && l > 0.f ? make_float2(kLowest, 0.f) : make_float2(m, l);
}
// 1 / L for a merged row: 0 of a row without keys (M = -inf)
CSA_DEVINL float inverse_sum(float M, float L) { return L > 0.f ? 1.0f / L : (M == -INFINITY ? 0.f : __int_as_float(0x7fffffff)); }

// Paged attention of a batch with a shared prefix (attend_prefix.cu): the query
// rows of the whole batch, [rows = n_bq * H][D], by tiles of 128, against tiles
// of 128 keys.  A row tile's units are the tiles of shared entries (read through
// the table's row 0) and of its requests' own keys; those of all row tiles are
// dealt to the CTA pairs in contiguous ranges, and a pair writes one partial per
// row tile that its range meets: partial p + r for pair p and row tile r,
// [rank 2][DP / 8 pieces][128 threads][4] fp32 with (running max in log2 units,
// sum) per row in ml.  O is not divided by the sum.
//
// Ranges are balanced by cost: a unit is 1, and a row tile begins with kPartCost
// more, what a pair spends on beginning and ending one (its rows, their norms,
// O to memory: ~10 us at D = 512 against 1.45 us a unit, 6 us against 0.9 at
// D = 128).  So a row tile's unit k lies kPartCost + k after its beginning.
// Few row tiles are not cut into as many ranges as there are pairs: with u units
// in each of R row tiles and r ranges per row tile a unit's time is spent u / r
// times, and the merge of r partials takes ~1/3 of it each, least at r =
// sqrt(3 u), that is at sqrt(3 u R * R) ranges (1 row tile of 130 units at D =
// 512: 57 us with 74 ranges, 40 us with 20).
struct PrefixPlan {
    static constexpr int kPartCost = 6;
    int row_tiles, pairs;
    CSA_HOSTDEV int partials() const { return pairs + row_tiles; }
    // the ranges that `units` units are cut into
    CSA_HOSTDEV int ranges(int units) const {
        const float r = sqrtf(3.f * (float)units * (float)row_tiles);
        return r < 1.f ? 1 : (r < (float)pairs ? (int)r : pairs);
    }
};

// Range p of n begins here: an even share of `total`, the first ones one more.
CSA_HOSTDEV inline int range_begin(int p, int n, int total) {
    const int each = total / n, more = total - each * n;
    return p >= n ? total : each * p + (p < more ? p : more);
}
// the range that holds place u
CSA_HOSTDEV inline int range_of(int u, int n, int total) {
    const int each = total / n, more = total - each * n;
    return u < more * (each + 1) ? u / (each + 1) : more + (u - more * (each + 1)) / each;
}

constexpr int kPrefixRows = 128, kPrefixKeys = 128;
CSA_HOSTDEV inline int prefix_dims(int D) { return D < 128 ? 128 : D; }  // a row's dims in the kernel (zero-padded)

struct PrefixArgs {
    AttendArgs a;          // of the whole call
    PrefixPlan plan;
    long long n_shared;
    // The entries' rows: the pool; or (own_cap >= 0) a bf16 copy of an FP8 cache: rows of the shared
    // entries in order, then own_cap rows of each request's own entries, then the rings
    const uint16_t *keys;
    int own_cap;
    uint16_t *hi, *lo;     // the query rows under gain, sign and RoPE as hi + lo (null: a.q itself),
    float *rq;             // and their factors (launch_query_rows)
    float *part;           // [partials][128][DP], see above
    float2 *ml;            // [partials][128]
    int2 *meet;            // [row_tiles] the first range that meets a row tile, and how many do (out)
};

PrefixPlan prefix_plan(long long rows);
int launch_query_rows(const PrefixArgs &p, cudaStream_t st);
int launch_expand_rows(const PrefixArgs &p, uint16_t *out, cudaStream_t st);  // that copy
int launch_attend_prefix(const PrefixArgs &p, const DevCtx &ctx, cudaStream_t st);

}  // namespace csa
