// gq4_kv_api.cu -- the extern "C" entry points between the QKV product and the
// output projection (declared in gq4.h): per-head norm and rotation, the
// paged 4-bit key/value cache and the attention over it.  As everywhere in
// the library, all checks run on the host before anything is enqueued.
#include <cstdint>

#include "gq4.h"
#include "gq4_checks.h"
#include "gq4_kv_internal.h"

namespace {

using gq4::aligned;
using gq4::RangeSet;

constexpr long long kMaxKeys = 1ll << 30;  // of one request: positions stay well inside 32 bits

// Rows x [T][heads][D], ld floats apart.
gq4_status check_rows(const float *x, int heads, int D, int ld)
{
    if (!x) return GQ4_ERR_INVALID_ARG;
    if (ld < heads * D || ld % 4 != 0) return GQ4_ERR_INVALID_ARG;
    if (!aligned(x, 16)) return GQ4_ERR_MISALIGNED;
    return GQ4_OK;
}

gq4_status check_cache(const gq4_kv_cache *c)
{
    if (!c) return GQ4_ERR_INVALID_ARG;
    if (c->n_pages <= 0 || c->kv_heads < 1 || c->kv_heads > GQ4_MAX_HEADS) return GQ4_ERR_INVALID_ARG;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
        return GQ4_ERR_INVALID_ARG;
    if ((long long)c->n_pages * c->page_size > 0x7fffffffll) return GQ4_ERR_INVALID_ARG;
    if (c->head_dim <= 0 || c->head_dim % 32 != 0) return GQ4_ERR_INVALID_ARG;
    if (c->group_size <= 0 || c->group_size % 32 != 0 || c->head_dim % c->group_size != 0)
        return GQ4_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128 && c->head_dim != 256)
        return GQ4_ERR_UNSUPPORTED;
    if (!c->Kq || !c->K_sz || !c->Vq || !c->V_sz) return GQ4_ERR_INVALID_ARG;
    if (!aligned(c->Kq, 16) || !aligned(c->K_sz, 16) || !aligned(c->Vq, 16) || !aligned(c->V_sz, 16))
        return GQ4_ERR_MISALIGNED;
    return GQ4_OK;
}

size_t cache_rows(const gq4_kv_cache *c)
{
    return (size_t)c->n_pages * (size_t)c->page_size * (size_t)c->kv_heads;
}

void cache_ranges(const gq4_kv_cache *c, bool written, RangeSet &rs)
{
    const size_t words = cache_rows(c) * (size_t)c->head_dim / 2;
    const size_t sz = cache_rows(c) * (size_t)(c->head_dim / c->group_size) * 8;
    const void *p[4] = {c->Kq, c->K_sz, c->Vq, c->V_sz};
    for (int i = 0; i < 4; ++i) {
        if (written)
            rs.output(p[i], i % 2 ? sz : words);
        else
            rs.input(p[i], i % 2 ? sz : words);
    }
}

gq4_status status_of(cudaError_t err)
{
    return err == cudaSuccess ? GQ4_OK : GQ4_ERR_CUDA;
}

// Both forms of the attention.
gq4_status attention(int B, int T, int q_heads, int max_pages, int max_query, int max_len, const gq4_kv_cache *cache,
                     const float *q, int ldq, const int32_t *query_start, const int32_t *seq_lens,
                     const int32_t *page_table, float scale, const gq4_kv_mask &mask, float *out, int ld_out,
                     void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    if (B < 1 || B > GQ4_MAX_REQUESTS || T < 0 || max_pages < 1 || max_query < 0 || max_len < 0 ||
        mask.window < 0 || mask.sinks < 0)
        return GQ4_ERR_INVALID_ARG;
    GQ4_TRY(check_cache(cache));
    if (q_heads < 1 || q_heads > GQ4_MAX_HEADS || q_heads % cache->kv_heads != 0)
        return GQ4_ERR_INVALID_ARG;
    const long long room = (long long)max_pages * cache->page_size;
    if (room > kMaxKeys) return GQ4_ERR_INVALID_ARG;
    if (!(scale - scale == 0.0f)) return GQ4_ERR_INVALID_ARG;  // NaN or infinite
    if (mask.tree && (mask.tree_words < 1 || mask.tree_words > GQ4_MAX_TREE_WORDS ||
                      (mask.window > 0 && !mask.positions)))
        return GQ4_ERR_INVALID_ARG;
    if (T == 0 || max_query == 0) return GQ4_OK;
    GQ4_TRY(check_rows(q, q_heads, cache->head_dim, ldq));
    GQ4_TRY(check_rows(out, q_heads, cache->head_dim, ld_out));
    if (!query_start || !seq_lens || !page_table) return GQ4_ERR_INVALID_ARG;
    if (!aligned(query_start, 4) || !aligned(seq_lens, 4) || !aligned(page_table, 4) ||
        !aligned(mask.tree, 4) || (mask.tree && mask.window > 0 && !aligned(mask.positions, 4)))
        return GQ4_ERR_MISALIGNED;
    const size_t need = gq4::attn_workspace_bytes(T, q_heads, cache->kv_heads, cache->head_dim, mask.tree != nullptr);
    if (!workspace || workspace_bytes < need) return GQ4_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return GQ4_ERR_MISALIGNED;
    const size_t width = (size_t)q_heads * cache->head_dim * 4;
    RangeSet rs;
    cache_ranges(cache, false, rs);
    rs.input_rows(q, T, width, (size_t)ldq * 4);
    rs.input(query_start, ((size_t)B + 1) * 4);
    rs.input(seq_lens, (size_t)B * 4);
    rs.input(page_table, (size_t)B * max_pages * 4);
    if (mask.tree) rs.input(mask.tree, (size_t)T * mask.tree_words * 4);
    if (mask.tree && mask.window > 0) rs.input(mask.positions, (size_t)T * 4);
    rs.output_rows(out, T, width, (size_t)ld_out * 4);
    rs.output(workspace, need);
    if (!rs.disjoint()) return GQ4_ERR_ALIAS;
    gq4::AttnCall c{};
    c.B = B;
    c.T = T;
    c.heads = q_heads;
    c.max_pages = max_pages;
    c.max_query = max_query;
    c.max_len = max_len > 0 && max_len < room ? max_len : (int)room;
    c.c = *cache;
    c.q = q;
    c.ldq = ldq;
    c.query_start = query_start;
    c.seq_lens = seq_lens;
    c.page_table = page_table;
    c.scale = scale;
    c.window = mask.window;
    // (first tokens count behind a window only)
    c.masks = mask.tree || (mask.window > 0 && mask.sinks > 0);
    c.sinks = mask.sinks < c.max_len ? mask.sinks : c.max_len;
    c.tree = mask.tree;
    c.tree_words = mask.tree_words;
    c.positions = mask.positions;
    c.out = out;
    c.ldo = ld_out;
    c.workspace = workspace;
    return status_of(gq4::launch_attn(c, stream));
}

// Both forms of the tree's bits and of accepting a path; slots: as planned
// (gq4_kv_tree_planned, gq4_kv_accept_planned).
gq4_status kv_tree(bool planned, int B, int T, int tree_words, int window, int sinks, const int32_t *parents,
                   const int32_t *slots, const int32_t *query_start, const int32_t *seq_lens, int32_t *positions,
                   uint32_t *tree, cudaStream_t stream)
{
    if (B < 1 || B > GQ4_MAX_REQUESTS || T < 0 || tree_words < 1 || tree_words > GQ4_MAX_TREE_WORDS ||
        window < 0 || sinks < 0)
        return GQ4_ERR_INVALID_ARG;
    if (T == 0) return GQ4_OK;
    if (!parents || !query_start || !seq_lens || !positions || !tree || (planned && !slots)) return GQ4_ERR_INVALID_ARG;
    const void *all[] = {parents, slots, query_start, seq_lens, positions, tree};
    for (const void *p : all)
        if (!aligned(p, 4)) return GQ4_ERR_MISALIGNED;
    RangeSet rs;
    rs.input(parents, (size_t)T * 4);
    rs.input(slots, (size_t)T * 4);
    rs.input(query_start, ((size_t)B + 1) * 4);
    rs.input(seq_lens, (size_t)B * 4);
    rs.output(positions, (size_t)T * 4);
    rs.output(tree, (size_t)T * tree_words * 4);
    if (!rs.disjoint()) return GQ4_ERR_ALIAS;
    gq4::TreeCall c{};
    c.B = B;
    c.T = T;
    c.words = tree_words;
    c.window = window;
    c.sinks = sinks;
    c.parents = parents;
    c.slots = slots;
    c.query_start = query_start;
    c.seq_lens = seq_lens;
    c.positions = positions;
    c.bits = tree;
    return status_of(gq4::launch_kv_tree(c, stream));
}

// (T < 0: without slots)
gq4_status kv_accept(int B, int T, int max_path, int max_pages, int n_free, const gq4_kv_cache *cache, const int32_t *path,
                     const int32_t *counts, const int32_t *slots, const int32_t *query_start, const int32_t *seq_lens,
                     const int32_t *page_table, int32_t *free_pages, const int32_t *free_count, int32_t *free_count_out,
                     int32_t *seq_lens_out, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    if (B < 1 || B > GQ4_MAX_REQUESTS || max_path < 0 || max_pages < 1 || n_free < 0)
        return GQ4_ERR_INVALID_ARG;
    GQ4_TRY(check_cache(cache));
    if ((long long)max_pages * cache->page_size > kMaxKeys) return GQ4_ERR_INVALID_ARG;
    if (!counts || !query_start || !seq_lens || !page_table || !free_count || !free_count_out || !seq_lens_out ||
        (n_free > 0 && !free_pages) || (T > 0 && !slots))
        return GQ4_ERR_INVALID_ARG;
    const void *all[] = {path, counts, slots, query_start, seq_lens, page_table, free_pages, free_count, free_count_out,
                         seq_lens_out};
    for (const void *p : all)
        if (!aligned(p, 4)) return GQ4_ERR_MISALIGNED;
    const size_t need = gq4_kv_accept_workspace_bytes(B), b = (size_t)B * 4;
    if (!workspace || workspace_bytes < need) return GQ4_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return GQ4_ERR_MISALIGNED;
    RangeSet rs;
    cache_ranges(cache, true, rs);
    rs.input(path, b * (size_t)max_path);
    rs.input(counts, b);
    if (T > 0) rs.input(slots, (size_t)T * 4);
    rs.input(query_start, b + 4);
    if (seq_lens_out != seq_lens) rs.input(seq_lens, b);
    rs.input(page_table, b * (size_t)max_pages);
    if (free_count_out != free_count) rs.input(free_count, 4);
    rs.output(free_pages, (size_t)n_free * 4);
    rs.output(free_count_out, 4);
    rs.output(seq_lens_out, b);
    rs.output(workspace, need);
    if (!rs.disjoint()) return GQ4_ERR_ALIAS;
    gq4::AcceptCall c{};
    c.B = B;
    c.T = T;
    c.max_path = max_path;
    c.max_pages = max_pages;
    c.n_free = n_free;
    c.c = *cache;
    c.path = path;
    c.counts = counts;
    c.slots = slots;
    c.query_start = query_start;
    c.seq_lens = seq_lens;
    c.page_table = page_table;
    c.free_count = free_count;
    c.free_pages = free_pages;
    c.free_count_out = free_count_out;
    c.seq_lens_out = seq_lens_out;
    c.verdict = static_cast<int32_t *>(workspace);
    return status_of(gq4::launch_kv_accept(c, stream));
}

}  // namespace

extern "C" {

gq4_status gq4_head_norm_rope(int T, int q_heads, int kv_heads, int head_dim, const gq4_rope *rope,
                              const int32_t *positions, const float *q, int ldq, const float *k,
                              int ldk, float *q_out, int ldq_out, float *k_out, int ldk_out,
                              cudaStream_t stream)
{
    if (!rope || T < 0 || q_heads < 0 || kv_heads < 0 || q_heads > GQ4_MAX_HEADS ||
        kv_heads > GQ4_MAX_HEADS || q_heads + kv_heads == 0)
        return GQ4_ERR_INVALID_ARG;
    if (head_dim < 8 || head_dim > GQ4_MAX_HEAD_DIM || head_dim % 8 != 0) return GQ4_ERR_INVALID_ARG;
    if (rope->rot_dim < 0 || rope->rot_dim > head_dim || rope->rot_dim % 8 != 0)
        return GQ4_ERR_INVALID_ARG;
    if (rope->interleaved != 0 && rope->interleaved != 1) return GQ4_ERR_INVALID_ARG;
    if (!(rope->eps >= 0.0f)) return GQ4_ERR_INVALID_ARG;  // also rejects NaN
    if (T == 0) return GQ4_OK;
    if (rope->rot_dim > 0 && (!positions || !rope->inv_freq)) return GQ4_ERR_INVALID_ARG;
    gq4::RopeCall c{};
    c.T = T;
    c.D = head_dim;
    c.rot = rope->rot_dim;
    c.interleaved = rope->interleaved != 0;
    c.eps = rope->eps;
    c.positions = positions;
    c.inv_freq = rope->inv_freq;
    const int heads[2] = {q_heads, kv_heads}, ldx[2] = {ldq, ldk}, ldy[2] = {ldq_out, ldk_out};
    const float *x[2] = {q, k}, *gain[2] = {rope->q_gain, rope->k_gain};
    float *y[2] = {q_out, k_out};
    RangeSet rs;
    if (rope->rot_dim > 0) {
        if (!aligned(positions, 4) || !aligned(rope->inv_freq, 4)) return GQ4_ERR_MISALIGNED;
        rs.input(positions, (size_t)T * 4);
        rs.input(rope->inv_freq, (size_t)rope->rot_dim / 2 * 4);
    }
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        GQ4_TRY(check_rows(x[i], heads[i], head_dim, ldx[i]));
        GQ4_TRY(check_rows(y[i], heads[i], head_dim, ldy[i]));
        if (gain[i] && !aligned(gain[i], 16)) return GQ4_ERR_MISALIGNED;
        const size_t width = (size_t)heads[i] * head_dim * 4;
        // in place: the same rows (each is read whole before it is written)
        if (!(x[i] == y[i] && ldx[i] == ldy[i])) rs.input_rows(x[i], T, width, (size_t)ldx[i] * 4);
        rs.output_rows(y[i], T, width, (size_t)ldy[i] * 4);
        rs.input(gain[i], (size_t)head_dim * 4);
        c.heads[i] = heads[i];
        c.x[i] = x[i];
        c.y[i] = y[i];
        c.gain[i] = gain[i];
        c.ldx[i] = ldx[i];
        c.ldy[i] = ldy[i];
    }
    if (!rs.disjoint()) return GQ4_ERR_ALIAS;
    return status_of(gq4::launch_rope(c, stream));
}

gq4_status gq4_kv_append(int T, const gq4_kv_cache *cache, const float *k, int ldk, const float *v,
                         int ldv, const int32_t *slots, cudaStream_t stream)
{
    if (T < 0) return GQ4_ERR_INVALID_ARG;
    GQ4_TRY(check_cache(cache));
    if (T == 0) return GQ4_OK;
    GQ4_TRY(check_rows(k, cache->kv_heads, cache->head_dim, ldk));
    GQ4_TRY(check_rows(v, cache->kv_heads, cache->head_dim, ldv));
    if (!slots) return GQ4_ERR_INVALID_ARG;
    if (!aligned(slots, 4)) return GQ4_ERR_MISALIGNED;
    const size_t width = (size_t)cache->kv_heads * cache->head_dim * 4;
    RangeSet rs;
    rs.input_rows(k, T, width, (size_t)ldk * 4);
    rs.input_rows(v, T, width, (size_t)ldv * 4);
    rs.input(slots, (size_t)T * 4);
    cache_ranges(cache, true, rs);
    if (!rs.disjoint()) return GQ4_ERR_ALIAS;
    return status_of(gq4::launch_kv_append(T, *cache, k, ldk, v, ldv, slots, stream));
}

gq4_status gq4_kv_rope_append(int T, int q_heads, const gq4_kv_cache *cache, const gq4_rope *rope,
                              const int32_t *positions, const float *q, int ldq, float *q_out,
                              int ldq_out, const float *k, int ldk, const float *v, int ldv,
                              const int32_t *slots, cudaStream_t stream)
{
    if (!rope || T < 0 || q_heads < 0 || q_heads > GQ4_MAX_HEADS) return GQ4_ERR_INVALID_ARG;
    GQ4_TRY(check_cache(cache));
    const int D = cache->head_dim;
    if (rope->rot_dim < 0 || rope->rot_dim > D || rope->rot_dim % 8 != 0) return GQ4_ERR_INVALID_ARG;
    if (rope->interleaved != 0 && rope->interleaved != 1) return GQ4_ERR_INVALID_ARG;
    if (!(rope->eps >= 0.0f)) return GQ4_ERR_INVALID_ARG;  // also rejects NaN
    if (T == 0) return GQ4_OK;
    if (rope->rot_dim > 0 && (!positions || !rope->inv_freq)) return GQ4_ERR_INVALID_ARG;
    GQ4_TRY(check_rows(k, cache->kv_heads, D, ldk));
    GQ4_TRY(check_rows(v, cache->kv_heads, D, ldv));
    if (!slots) return GQ4_ERR_INVALID_ARG;
    if (!aligned(slots, 4)) return GQ4_ERR_MISALIGNED;
    const size_t width = (size_t)cache->kv_heads * D * 4;
    RangeSet rs;
    if (rope->rot_dim > 0) {
        if (!aligned(positions, 4) || !aligned(rope->inv_freq, 4)) return GQ4_ERR_MISALIGNED;
        rs.input(positions, (size_t)T * 4);
        rs.input(rope->inv_freq, (size_t)rope->rot_dim / 2 * 4);
    }
    if (rope->k_gain && !aligned(rope->k_gain, 16)) return GQ4_ERR_MISALIGNED;
    gq4::RopeCall c{};
    c.T = T;
    c.D = D;
    c.rot = rope->rot_dim;
    c.interleaved = rope->interleaved != 0;
    c.eps = rope->eps;
    c.positions = positions;
    c.inv_freq = rope->inv_freq;
    c.x[1] = k;
    c.ldx[1] = ldk;
    c.gain[1] = rope->k_gain;
    if (q_heads > 0) {
        GQ4_TRY(check_rows(q, q_heads, D, ldq));
        GQ4_TRY(check_rows(q_out, q_heads, D, ldq_out));
        if (rope->q_gain && !aligned(rope->q_gain, 16)) return GQ4_ERR_MISALIGNED;
        const size_t q_width = (size_t)q_heads * D * 4;
        // in place: the same rows (each is read whole before it is written)
        if (!(q == q_out && ldq == ldq_out)) rs.input_rows(q, T, q_width, (size_t)ldq * 4);
        rs.output_rows(q_out, T, q_width, (size_t)ldq_out * 4);
        rs.input(rope->q_gain, (size_t)D * 4);
        c.heads[0] = q_heads;
        c.x[0] = q;
        c.y[0] = q_out;
        c.gain[0] = rope->q_gain;
        c.ldx[0] = ldq;
        c.ldy[0] = ldq_out;
    }
    rs.input_rows(k, T, width, (size_t)ldk * 4);
    rs.input_rows(v, T, width, (size_t)ldv * 4);
    rs.input(rope->k_gain, (size_t)D * 4);
    rs.input(slots, (size_t)T * 4);
    cache_ranges(cache, true, rs);
    if (!rs.disjoint()) return GQ4_ERR_ALIAS;
    return status_of(gq4::launch_kv_rope_append(c, *cache, v, ldv, slots, stream));
}

gq4_status gq4_kv_gather(int T, const gq4_kv_cache *cache, const int32_t *slots, float *k_out,
                         float *v_out, cudaStream_t stream)
{
    if (T < 0) return GQ4_ERR_INVALID_ARG;
    GQ4_TRY(check_cache(cache));
    if (T == 0) return GQ4_OK;
    if (!slots || !k_out || !v_out) return GQ4_ERR_INVALID_ARG;
    if (!aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16)) return GQ4_ERR_MISALIGNED;
    const size_t bytes = (size_t)T * cache->kv_heads * cache->head_dim * 4;
    RangeSet rs;
    cache_ranges(cache, false, rs);
    rs.input(slots, (size_t)T * 4);
    rs.output(k_out, bytes);
    rs.output(v_out, bytes);
    if (!rs.disjoint()) return GQ4_ERR_ALIAS;
    return status_of(gq4::launch_kv_gather(T, *cache, slots, k_out, v_out, stream));
}

gq4_status gq4_kv_plan(int B, int T, int page_size, int max_pages, int n_free,
                       const int32_t *past_lens, const int32_t *new_lens, int32_t *page_table,
                       const int32_t *free_pages, const int32_t *free_count,
                       int32_t *free_count_out, int32_t *seq_lens, int32_t *query_start,
                       int32_t *positions, int32_t *slots, cudaStream_t stream)
{
    if (B < 1 || B > GQ4_MAX_REQUESTS || T < 0 || max_pages < 1 || n_free < 0)
        return GQ4_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0)
        return GQ4_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size > kMaxKeys) return GQ4_ERR_INVALID_ARG;
    if (!past_lens || !new_lens || !page_table || !free_count || !free_count_out || !seq_lens ||
        !query_start || (T > 0 && (!positions || !slots)) || (n_free > 0 && !free_pages))
        return GQ4_ERR_INVALID_ARG;
    const void *all[] = {past_lens, new_lens, page_table, free_pages, free_count, free_count_out,
                         seq_lens, query_start, positions, slots};
    for (const void *p : all)
        if (!aligned(p, 4)) return GQ4_ERR_MISALIGNED;
    const size_t b = (size_t)B * 4, t = (size_t)T * 4;
    RangeSet rs;
    if (seq_lens != past_lens) rs.input(past_lens, b);
    rs.input(new_lens, b);
    rs.input(free_pages, (size_t)n_free * 4);
    if (free_count_out != free_count) rs.input(free_count, 4);
    rs.output(page_table, b * (size_t)max_pages);
    rs.output(free_count_out, 4);
    rs.output(seq_lens, b);
    rs.output(query_start, b + 4);
    rs.output(positions, t);
    rs.output(slots, t);
    if (!rs.disjoint()) return GQ4_ERR_ALIAS;
    gq4::PlanCall c{};
    c.B = B;
    c.T = T;
    c.page = page_size;
    c.max_pages = max_pages;
    c.n_free = n_free;
    c.past_lens = past_lens;
    c.new_lens = new_lens;
    c.free_pages = free_pages;
    c.free_count = free_count;
    c.page_table = page_table;
    c.free_count_out = free_count_out;
    c.seq_lens = seq_lens;
    c.query_start = query_start;
    c.positions = positions;
    c.slots = slots;
    return status_of(gq4::launch_kv_plan(c, stream));
}

gq4_status gq4_kv_tree(int B, int T, int tree_words, int window, int sinks, const int32_t *parents,
                       const int32_t *query_start, const int32_t *seq_lens, int32_t *positions,
                       uint32_t *tree, cudaStream_t stream)
{
    return kv_tree(false, B, T, tree_words, window, sinks, parents, nullptr, query_start, seq_lens, positions, tree, stream);
}

gq4_status gq4_kv_tree_planned(int B, int T, int tree_words, int window, int sinks, const int32_t *parents,
                               const int32_t *slots, const int32_t *query_start, const int32_t *seq_lens,
                               int32_t *positions, uint32_t *tree, cudaStream_t stream)
{
    return kv_tree(true, B, T, tree_words, window, sinks, parents, slots, query_start, seq_lens, positions, tree, stream);
}

size_t gq4_kv_accept_workspace_bytes(int B)
{
    return B < 1 ? 0 : ((size_t)B * 4 + 255) / 256 * 256;
}

gq4_status gq4_kv_accept(int B, int max_path, int max_pages, int n_free, const gq4_kv_cache *cache,
                         const int32_t *path, const int32_t *counts, const int32_t *query_start,
                         const int32_t *seq_lens, const int32_t *page_table, int32_t *free_pages,
                         const int32_t *free_count, int32_t *free_count_out, int32_t *seq_lens_out,
                         void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    return kv_accept(B, -1, max_path, max_pages, n_free, cache, path, counts, nullptr, query_start, seq_lens, page_table,
                     free_pages, free_count, free_count_out, seq_lens_out, workspace, workspace_bytes, stream);
}

gq4_status gq4_kv_accept_planned(int B, int T, int max_path, int max_pages, int n_free, const gq4_kv_cache *cache,
                                 const int32_t *path, const int32_t *counts, const int32_t *slots,
                                 const int32_t *query_start, const int32_t *seq_lens, const int32_t *page_table,
                                 int32_t *free_pages, const int32_t *free_count, int32_t *free_count_out,
                                 int32_t *seq_lens_out, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    if (T < 0) return GQ4_ERR_INVALID_ARG;
    return kv_accept(B, T, max_path, max_pages, n_free, cache, path, counts, slots, query_start, seq_lens, page_table,
                     free_pages, free_count, free_count_out, seq_lens_out, workspace, workspace_bytes, stream);
}

size_t gq4_kv_attention_workspace_bytes(int T, int q_heads, int kv_heads, int head_dim)
{
    if (T < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1) return 0;
    return gq4::attn_workspace_bytes(T, q_heads, kv_heads, head_dim, false);
}

size_t gq4_kv_attention_masked_workspace_bytes(int T, int q_heads, int kv_heads, int head_dim)
{
    if (T < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1) return 0;
    return gq4::attn_workspace_bytes(T, q_heads, kv_heads, head_dim, true);
}

gq4_status gq4_kv_attention(int B, int T, int q_heads, int max_pages, int max_query, int max_len,
                            const gq4_kv_cache *cache, const float *q, int ldq,
                            const int32_t *query_start, const int32_t *seq_lens,
                            const int32_t *page_table, float scale, int window, float *out,
                            int ld_out, void *workspace, size_t workspace_bytes,
                            cudaStream_t stream)
{
    gq4_kv_mask mask{};
    mask.window = window;
    return attention(B, T, q_heads, max_pages, max_query, max_len, cache, q, ldq, query_start, seq_lens, page_table, scale,
                     mask, out, ld_out, workspace, workspace_bytes, stream);
}

gq4_status gq4_kv_attention_masked(int B, int T, int q_heads, int max_pages, int max_query, int max_len,
                                   const gq4_kv_cache *cache, const float *q, int ldq,
                                   const int32_t *query_start, const int32_t *seq_lens,
                                   const int32_t *page_table, float scale, const gq4_kv_mask *mask,
                                   float *out, int ld_out, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream)
{
    if (!mask) return GQ4_ERR_INVALID_ARG;
    return attention(B, T, q_heads, max_pages, max_query, max_len, cache, q, ldq, query_start, seq_lens, page_table, scale,
                     *mask, out, ld_out, workspace, workspace_bytes, stream);
}

}  // extern "C"
