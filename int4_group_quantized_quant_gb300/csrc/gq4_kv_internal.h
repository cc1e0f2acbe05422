// gq4_kv_internal.h -- the launches behind the entry points between the QKV
// product and the output projection: rotation, cache, attention.
#pragma once

#include "gq4_internal.h"

namespace gq4 {

// Per-head norm and rotation (gq4_head_norm_rope).  A side with 0 heads is
// absent.
struct RopeCall {
    int T, D, rot;
    bool interleaved;
    int heads[2];          // q, k
    const float *x[2];
    float *y[2];
    const float *gain[2];  // NULL: not normalised
    int ldx[2], ldy[2];
    float eps;
    const int32_t *positions;
    const float *inv_freq;
};
cudaError_t launch_rope(const RopeCall &call, cudaStream_t stream);

// The paged 4-bit key/value cache: writer, reader, a step's book-keeping.
cudaError_t launch_kv_append(int T, const gq4_kv_cache &c, const float *k, int ldk, const float *v,
                             int ldv, const int32_t *slots, cudaStream_t stream);
cudaError_t launch_kv_gather(int T, const gq4_kv_cache &c, const int32_t *slots, float *k_out,
                             float *v_out, cudaStream_t stream);
struct PlanCall {
    int B, T, page, max_pages, n_free;
    const int32_t *past_lens, *new_lens, *free_pages, *free_count;
    int32_t *page_table, *free_count_out, *seq_lens, *query_start, *positions, *slots;
};
cudaError_t launch_kv_plan(const PlanCall &call, cudaStream_t stream);
cudaError_t read_kv_device_error(unsigned int *bits, bool clear);
// Rotation and append in one: side 1 of the call is k, which has no output.
cudaError_t launch_kv_rope_append(const RopeCall &call, const gq4_kv_cache &c, const float *v, int ldv,
                                  const int32_t *slots, cudaStream_t stream);
cudaError_t read_kv_rope_device_error(unsigned int *bits, bool clear);

// Drafted trees: their bits, and accepting a path.
struct TreeCall {
    int B, T, words, window, sinks;
    const int32_t *parents, *slots, *query_start, *seq_lens;   // slots: as planned, or NULL
    int32_t *positions;
    uint32_t *bits;
};
cudaError_t launch_kv_tree(const TreeCall &call, cudaStream_t stream);
struct AcceptCall {
    int B, max_path, max_pages, n_free;
    gq4_kv_cache c;
    const int32_t *path, *counts, *query_start, *seq_lens, *page_table, *free_count;
    int32_t *free_pages, *free_count_out, *seq_lens_out;
    int32_t *verdict;   // [B] of the workspace: how many rows, -1: refused
    const int32_t *slots;   // [T] as planned
    int T;              // -1: there are none
};
cudaError_t launch_kv_accept(const AcceptCall &call, cudaStream_t stream);
cudaError_t read_tree_device_error(unsigned int *bits, bool clear);

// Attention over the cache.
constexpr int kPromptTile = 128, kPromptKeys = 64;   // query rows and keys of a tile of the prompt kernel
// What a row tile of the prompt kernel leaves to the call's last kernel: a bit
// per row, and whether to look for rows that see small values only.
struct ApartTile {
    uint32_t rows[kPromptTile / 32];
    int request, tile, uneven, unused;
};
constexpr int kUndone = -2;
struct AttnCall {
    int B, T, heads, max_pages, max_query, max_len;
    gq4_kv_cache c;
    const float *q;
    int ldq;
    const int32_t *query_start, *seq_lens, *page_table;
    float scale;
    int window;
    bool masks;             // the masked form: what follows counts
    int sinks;              // first keys that a window does not hide
    const uint32_t *tree;   // ancestor bits [T][tree_words], or NULL
    int tree_words;
    const int32_t *positions;   // [T], with bits and a window
    float *out;
    int ldo;
    void *workspace;
    int prompt_rows;   // requests of at least so many query rows per kv head go to the prompt kernel
    ApartTile *apart;  // in the workspace, one for each of the prompt kernel's CTAs
    long long n_apart;
    // Trees: the prompt kernel's CTAs share the tiles (gq4_attn_prompt.cuh).  Marks 0 .. n_units - 1 are then the row
    // tiles', behind them two for each CTA's sums of row tiles that are cut.
    int tree_ctas;
    long long n_units;
    float *pieces;     // [tree_ctas][2][kPromptTile][D + 2] sums: the rows', then the maximum and the weights' sum of each
    int4 *cut;         // [tree_ctas] the row tile that starts in the CTA and is cut: request, tile, kv head, last CTA or -1
                       // (kUndone: the CTA gave up before it had done its share)
};
size_t attn_workspace_bytes(int T, int heads, int kv_heads, int D, bool masks);
cudaError_t launch_attn(const AttnCall &call, cudaStream_t stream);
cudaError_t read_attn_device_error(unsigned int *bits, bool clear);
// Its kernel for requests with many query rows.
bool prompt_path_supported(const AttnCall &call);
cudaError_t launch_attn_prompt(const AttnCall &call, cudaStream_t stream);
cudaError_t read_prompt_device_error(unsigned int *bits, bool clear);
// Both kernels' masked forms.
cudaError_t launch_attn_masked(const AttnCall &call, cudaStream_t stream);
cudaError_t read_masked_device_error(unsigned int *bits, bool clear);
cudaError_t launch_attn_prompt_masked(const AttnCall &call, cudaStream_t stream);
cudaError_t read_prompt_masked_device_error(unsigned int *bits, bool clear);
cudaError_t launch_attn_prompt_tree(const AttnCall &call, cudaStream_t stream);
cudaError_t read_prompt_tree_device_error(unsigned int *bits, bool clear);

}  // namespace gq4
