// For tests/test_gpu_undone.py: the last kernel of a tree call alone, over the workspace that a call has left.
#include "gq4_attn_split.cuh"

extern "C" __attribute__((visibility("default")))
int run_join(int B, int T, int heads, int max_pages, int max_query, int max_len, const gq4_kv_cache *cache, const float *q, int ldq,
             const int *query_start, const int *seq_lens, const int *page_table, float scale, const uint32_t *tree, int words,
             float *out, int ldo, int least, void *apart, long long n_units, int ctas, void *cut, float *pieces,
             cudaStream_t stream)
{
    if (cache->head_dim != 128 || cache->group_size != 128) return -1;
    gq4::SplitParams p{};
    gq4::AttnCall &a = p.a;
    a.B = B;
    a.T = T;
    a.heads = heads;
    a.max_pages = max_pages;
    a.max_query = max_query;
    a.max_len = max_len;
    a.c = *cache;
    a.q = q;
    a.ldq = ldq;
    a.query_start = query_start;
    a.seq_lens = seq_lens;
    a.page_table = page_table;
    a.scale = scale;
    a.masks = true;
    a.tree = tree;
    a.tree_words = words;
    a.out = out;
    a.ldo = ldo;
    a.prompt_rows = least;
    a.apart = static_cast<gq4::ApartTile *>(apart);
    a.n_units = n_units;
    a.n_apart = n_units + 2 * ctas;
    a.tree_ctas = ctas;
    a.cut = static_cast<int4 *>(cut);
    a.pieces = pieces;
    p.R = heads / cache->kv_heads;
    p.grid = 0;     // (no sums of the kernel for few rows)
    gq4::attn_join_kernel<8, 4, 1, true><<<ctas * gq4::kPieceParts, gq4::kJoinThreads, 0, stream>>>(p, 128);
    return (int)cudaGetLastError();
}

// Where a call's marks begin in its workspace (heads of 128).
extern "C" __attribute__((visibility("default")))
long long sums_bytes()
{
    return 2ll * gq4::kMaxGrid * sizeof(int4) + 4ll * gq4::kMaxGrid * (2 + gq4::kWarps) * (128 + 2) * sizeof(float);
}
