// gq4_attn_masked.cu -- the kernel for few rows behind first tokens that stay
// visible and with ancestor bits (gq4_kv_attention_masked).
#include "gq4_attn_split.cuh"

namespace gq4 {

cudaError_t launch_attn_masked(const AttnCall &call, cudaStream_t stream)
{
    return launch_few_rows<true>(call, stream);
}

cudaError_t read_masked_device_error(unsigned int *bits, bool clear)
{
    return read_split_error(bits, clear);
}

}  // namespace gq4
