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

size_t sums_bytes(int D)
{
    // rows of sums of all CTAs: 304 of 8 rows at 64 dims, above that 304 of 4 or 152 of 8
    const size_t rows = D <= 64 ? kMaxGrid * 8 : kMaxGrid * 4;
    return 2 * kMaxGrid * sizeof(int4) + rows * (2 + kWarps) * (size_t)(D + 2) * sizeof(float);
}

}  // namespace

size_t attn_workspace_bytes(int T, int heads, int kv_heads, int D)
{
    static_assert(sizeof(ApartTile) == 32, "a multiple of 16 bytes");
    return sums_bytes(D) + (size_t)prompt_ctas(GQ4_MAX_REQUESTS, T, heads, kv_heads) * sizeof(ApartTile);
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
    const bool prompt = prompt_path_supported(call) && call.max_query * R >= kPromptRows &&
                        (long long)call.T * call.heads >= kPromptTotal;
    call.prompt_rows = prompt ? kPromptRows : 0x7fffffff;
    call.apart = reinterpret_cast<ApartTile *>(static_cast<char *>(call.workspace) + sums_bytes(call.c.head_dim));
    call.n_apart = prompt ? prompt_ctas(call.B, call.T, call.heads, call.c.kv_heads) : 0;
    if (prompt) {
        const cudaError_t err = call.masks ? launch_attn_prompt_masked(call, stream) : launch_attn_prompt(call, stream);
        if (err != cudaSuccess) return err;
    }
    return call.masks ? launch_attn_masked(call, stream) : launch_few_rows<false>(call, stream);
}

cudaError_t read_attn_device_error(unsigned int *bits, bool clear)
{
    cudaError_t (*const words[])(unsigned int *, bool) = {read_split_error, read_masked_device_error, read_prompt_device_error,
                                                          read_prompt_masked_device_error};
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
