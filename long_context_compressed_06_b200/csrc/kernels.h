// kernels.h -- internal host-side launchers (validated arguments in, status out).
// The C ABI in abi.cu validates every argument and then calls these.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace csa {

struct DevCtx;

int launch_compress(const uint16_t *A, const uint16_t *B, const float *logits, int batch, long long T,
                    int d, int m, int apply_rmsnorm, const float *gain, float eps, uint16_t *out,
                    cudaStream_t st);

int launch_compress_dynamic(const uint16_t *A, const uint16_t *B, const uint16_t *Za, const uint16_t *Zb,
                            const float *bias, int batch, long long T, int d, int m, int apply_rmsnorm,
                            const float *gain, float eps, long long i0, long long ni, long long n_out,
                            uint16_t *out, cudaStream_t st);

int launch_quantize_fp8_kv(const uint16_t *x, long long rows, int d, uint8_t *codes, uint8_t *exps, cudaStream_t st);

int launch_index(const uint16_t *q_idx, const float *w, const uint16_t *k_idx, const int *q_pos,
                 int batch, int nq, long long N, int H_I, int d_I, int m, float *scores,
                 const DevCtx &ctx, cudaStream_t st);

int launch_quantize_fp4(const uint16_t *x, long long rows, int d, uint8_t *packed, uint8_t *scales,
                        cudaStream_t st);

int launch_index_fp4(const uint8_t *q4, const uint8_t *q4s, const float *w, const uint8_t *k4,
                     const uint8_t *k4s, const int *q_pos, int batch, int nq, long long N, int H_I,
                     int d_I, int m, float *scores, const DevCtx &ctx, cudaStream_t st);

size_t topk_workspace_bytes(int batch, int nq, long long N, int k);
// q_pos may be null inside the library: every entry is then eligible.
// pdl: launched as a programmatic dependent of the stream's previous kernel
// (the kernel waits for it before reading scores) -- only for chains whose
// predecessor is this library's own kernel (csa_decode_step).
int launch_topk(const float *scores, const int *q_pos, int batch, int nq, long long N, int m, int k,
                int *idx, cudaStream_t st, bool pdl = false);

size_t rescore_workspace_bytes(int batch, int nq, int kc, int k, int d_I);
bool rescore_supported(int H_I, int d_I);
int launch_rescore_topk(const uint16_t *q_idx, const float *w, const uint16_t *k_idx, const int *cand, int kc,
                        int batch, int nq, long long N, int H_I, int d_I, int k, int *idx, void *ws,
                        const DevCtx &ctx, cudaStream_t st);

// Shapes the tensor-core indexers take (the only implementation).
bool index_tc_supported(int H_I, int d_I);
bool index_fp4_tc_supported(int H_I, int d_I);
int launch_index_tc(const uint16_t *q_idx, const float *w, const uint16_t *k_idx, const int *q_pos, int batch,
                    int nq, long long N, int H_I, int d_I, int m, float *scores, const DevCtx &ctx,
                    cudaStream_t st);

// Attention: dense selects the HCA key set of the first n_vis(t) entries;
// otherwise the k selected entries idx (may be null when k == 0).
size_t attend_workspace_bytes(int batch, int nq, int H, int D, long long max_keys);
// The FP8 KV cache of one attention call: e4m3 codes and UE8M0 exponent
// bytes of the compressed entries and of the window rows.
struct Fp8Kv {
    const uint8_t *kv, *kv_exp, *win, *win_exp;
};

int launch_attend(const uint16_t *q, const float *q_gain, const float *sinks, const float *rope_cos,
                  const float *rope_sin, long long rope_npos, const Fp8Kv *fp8, const uint16_t *kv, long long N, int m,
                  const int *idx, int k, bool dense, const uint16_t *win, long long win_pos0, long long win_rows,
                  int W, const int *q_pos,
                  int batch, int nq, int H, int D, float scale, float eps, uint16_t *out,
                  void *ws, size_t ws_bytes, const DevCtx &ctx, cudaStream_t st, bool pdl = false);

// Attention over a paged cache (csa_paged / hca_attend_paged): the arguments
// of one call, bf16 rows (pool, ring) or FP8 rows (fp8: kv / win fields).
struct PagedArgs {
    const uint16_t *q;
    const float *q_gain, *sinks, *rope_cos, *rope_sin;
    long long rope_npos;
    const uint16_t *pool;  // [n_pages][page][D]
    Fp8Kv fp8;             // or its codes and exponents (fp8.kv set)
    long long n_pages;
    int page;
    const int *table;      // [batch][max_pages]
    int max_pages;
    long long n_shared;    // leading entries that every row of the table shares
    int m;
    const uint16_t *ring;  // [batch][ring_rows][D]
    int ring_rows, W;
    const int *q_pos;
    int batch, nq, H, D;
    float scale, eps;
    uint16_t *out;
};

size_t attend_paged_workspace_bytes(int batch, int nq, int H, int D, int page, int max_pages, long long n_shared,
                                    int ring_rows, int W, bool fp8, bool rewrite);
inline bool paged_rewrite(const PagedArgs &a) { return a.q_gain || a.rope_cos || a.scale < 0.f; }
int launch_attend_paged(const PagedArgs &a, void *ws, size_t ws_bytes, const DevCtx &ctx, cudaStream_t st);

// Block tables and slot maps (csa_plan_pages); the pointers' shapes are the ABI's.
struct PlanArgs {
    const int *old_len, *new_len;
    int batch, m, page, ring;
    const int *free_pages;
    long long n_free;
    int *table;
    int max_pages;
    long long *cu_tokens, *cu_entries, *cu_pages;  // cu_pages: workspace (large batches)
    long long *entry_slots;
    long long max_entries;
    int *tok_pos;
    long long *win_slots;
    long long max_tokens;
    long long *counts;
};

size_t plan_workspace_bytes(int batch);
int launch_plan_pages(const PlanArgs &a, void *ws, cudaStream_t st);

// rows [n][d] to rows slots[i] of pool (bf16) or of codes / exps (FP8 rows, codes set)
int launch_paged_write(const uint16_t *rows, const long long *slots, long long n, int d, uint16_t *pool, uint8_t *codes,
                       uint8_t *exps, long long n_slots, cudaStream_t st);

int launch_selftest_wait(const DevCtx &ctx, cudaStream_t st);

// Host-side argument checks of csa_attend (everything but the workspace).
int check_attend_args(const uint16_t *q, const float *q_gain, const float *sinks, const float *rope_cos,
                      const float *rope_sin, long long rope_positions, const uint16_t *kv, long long N,
                      const int *idx, int k, const uint16_t *win, long long win_pos0, long long win_rows, int W,
                      const int *q_pos, int batch, int nq, int H, int D, float eps, const void *out);

}  // namespace csa
