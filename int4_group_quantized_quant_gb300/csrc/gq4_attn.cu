// gq4_attn.cu -- attention over the paged 4-bit key/value cache: which kernels
// a call takes, its workspace, and the causal form of the kernel for few rows.
#include "gq4_attn_split.cuh"

namespace gq4 {
namespace {

// Requests of at least so many query rows per kv head, and calls of so many
// rows in all, are the prompt kernel's.
constexpr int kPromptRows = 48, kPromptTotal = 5120;

// The prompt kernel's CTAs: as many row tiles as its requests can have
// together, per kv head.
long long prompt_ctas(int B, int T, int heads, int kv_heads)
{
    const long long rows = (long long)T * (heads / kv_heads), most = rows / kPromptRows;
    return ((rows + kPromptTile - 1) / kPromptTile + (B < most ? B : most)) * kv_heads;
}

// Trees: requests of at least so many query rows per kv head (of one scale group
// per row, of several), and calls of so many scores in all.
constexpr int kTreeRows[2] = {64, 96};
constexpr long long kTreeScores = 8 << 20;
// The CTAs that share the tiles of a tree call, at most.
constexpr int kTreeCtas = 152;

size_t tree_bytes(int D)
{
    return D > 128 ? 0 : kTreeCtas * (2 * sizeof(ApartTile) + sizeof(int4) + 2 * (size_t)kPromptTile * (D + 2) * sizeof(float));
}

size_t sums_bytes(int D)
{
    // rows of sums of all CTAs: 304 of 8 rows at 64 dims, above that 304 of 4 or 152 of 8
    const size_t rows = D <= 64 ? kMaxGrid * 8 : kMaxGrid * 4;
    return 2 * kMaxGrid * sizeof(int4) + rows * (2 + kWarps) * (size_t)(D + 2) * sizeof(float);
}

}  // namespace

size_t attn_workspace_bytes(int T, int heads, int kv_heads, int D, bool masks)
{
    static_assert(sizeof(ApartTile) == 32, "a multiple of 16 bytes");
    return sums_bytes(D) + (size_t)prompt_ctas(GQ4_MAX_REQUESTS, T, heads, kv_heads) * sizeof(ApartTile) +
           (masks && (long long)T * (heads / kv_heads) >= kTreeRows[0] ? tree_bytes(D) : 0);
}

cudaError_t launch_attn(const AttnCall &in, cudaStream_t stream)
{
    // Requests of many query rows go to the prompt kernel, whose tiles hold
    // 128 rows, if there are enough rows in all to fill its CTAs.  Measured
    // with 4096 keys and more behind 32 heads over 8 of 128, one group:
    // 16 requests of 8 tokens (32 rows each, 4096 in all) 88 us there and 83
    // here, of 12 (48, 6144) 88 and 116, of 16 89 and 150; one request of 64
    // tokens (256, 2048) 90 and 50.  Four groups: of 12 169 and 150, of 16
    // 170 and 197.  (Measured at this shape only; with four groups the border
    // lies somewhat higher, and few rows behind a long past leave SMs idle.)
    AttnCall call = in;
    const long long R = call.heads / call.c.kv_heads;
    // Trees, whose tiles all CTAs share there, by their scores, rows times keys.
    // 32 heads over 8 of 128, one group, few-rows kernel / prompt kernel: one
    // request of 26 nodes 31 / 39 us behind 4000 keys and 70 / 49 behind 16000;
    // 4 of them 33 / 43 behind 1000 and 72 / 49 behind 4000; 16 of 12 nodes (48
    // rows) 70 / 70 behind 2000, of 16 89 / 72, 48 of 9 93 / 115 behind 1000.
    // Several groups: 16 of 16 99 / 103 behind 2000, 4 of 26 80 / 64 behind 4000.
    const bool one = call.c.head_dim == call.c.group_size;
    const int least = call.tree ? kTreeRows[one ? 0 : 1] : kPromptRows;
    const long long seen = call.tree && call.window > 0 ? (long long)call.window + call.sinks + call.max_query : call.max_len;
    const bool enough = call.tree ? (long long)call.T * call.heads * (seen < call.max_len ? seen : call.max_len) >= kTreeScores
                                  : (long long)call.T * call.heads >= kPromptTotal;
    // (the workspace of a tree call goes by T: no request has more rows than that)
    const long long most = call.tree && call.T < call.max_query ? call.T : call.max_query;
    const bool prompt = prompt_path_supported(call) && most * R >= least && enough;
    call.prompt_rows = prompt ? least : 0x7fffffff;
    call.apart = reinterpret_cast<ApartTile *>(static_cast<char *>(call.workspace) + sums_bytes(call.c.head_dim));
    call.n_units = call.n_apart = prompt ? prompt_ctas(call.B, call.T, call.heads, call.c.kv_heads) : 0;
    call.tree_ctas = 0;
    if (prompt && call.tree) {
        int dev = 0, sms = 0;
        cudaError_t err;
        if ((err = cudaGetDevice(&dev)) != cudaSuccess ||
            (err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return err;
        call.tree_ctas = sms < kTreeCtas ? sms : kTreeCtas;
        call.n_apart += 2 * call.tree_ctas;
        call.cut = reinterpret_cast<int4 *>(call.apart + call.n_apart);
        call.pieces = reinterpret_cast<float *>(call.cut + call.tree_ctas);
    }
    if (prompt) {
        const cudaError_t err = call.tree    ? launch_attn_prompt_tree(call, stream)
                                : call.masks ? launch_attn_prompt_masked(call, stream)
                                             : launch_attn_prompt(call, stream);
        if (err != cudaSuccess) return err;
    }
    return call.masks ? launch_attn_masked(call, stream) : launch_few_rows<false>(call, stream);
}

cudaError_t read_attn_device_error(unsigned int *bits, bool clear)
{
    cudaError_t (*const words[])(unsigned int *, bool) = {read_split_error, read_masked_device_error, read_prompt_device_error,
                                                          read_prompt_masked_device_error, read_prompt_tree_device_error};
    *bits = 0;
    for (auto read : words) {
        unsigned int more = 0;
        const cudaError_t err = read(&more, clear);
        if (err != cudaSuccess) return err;
        *bits |= more;
    }
    return cudaSuccess;
}

}  // namespace gq4
