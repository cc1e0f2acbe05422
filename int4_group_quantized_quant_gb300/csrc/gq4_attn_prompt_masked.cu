// gq4_attn_prompt_masked.cu -- the kernel for many rows behind first tokens that
// stay visible (gq4_kv_attention_masked).
#include "gq4_attn_prompt.cuh"

namespace gq4 {

cudaError_t launch_attn_prompt_masked(const AttnCall &call, cudaStream_t stream)
{
    return launch_many_rows<kSinks>(call, stream);
}

cudaError_t read_prompt_masked_device_error(unsigned int *bits, bool clear)
{
    return read_prompt_error(bits, clear);
}

}  // namespace gq4
