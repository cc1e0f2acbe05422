// gq4_attn_prompt.cu -- the kernel for many rows in its causal form.
#include "gq4_attn_prompt.cuh"

namespace gq4 {

bool prompt_path_supported(const AttnCall &call)
{
    return call.c.head_dim <= 128;
}

cudaError_t launch_attn_prompt(const AttnCall &call, cudaStream_t stream)
{
    return launch_many_rows<kCausal>(call, stream);
}

cudaError_t read_prompt_device_error(unsigned int *bits, bool clear)
{
    return read_prompt_error(bits, clear);
}

}  // namespace gq4
