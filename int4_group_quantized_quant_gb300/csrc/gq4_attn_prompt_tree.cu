// gq4_attn_prompt_tree.cu -- the kernel for many rows with ancestor bits (gq4_kv_attention_masked).
#include "gq4_attn_prompt.cuh"

namespace gq4 {

cudaError_t launch_attn_prompt_tree(const AttnCall &call, cudaStream_t stream)
{
    return launch_many_rows<kTree>(call, stream);
}

cudaError_t read_prompt_tree_device_error(unsigned int *bits, bool clear)
{
    return read_prompt_error(bits, clear);
}

}  // namespace gq4
