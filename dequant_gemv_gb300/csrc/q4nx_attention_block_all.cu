// q4nx_attention_block_all.cu -- the kernel for many query rows, all positions.
#include "q4nx_attention_block.cuh"

namespace q4nx {

template cudaError_t launch_attention_block<kAll>(int, const AttnArgsOf<kAll>&, int64_t, int, int, const DeviceInfo&, cudaStream_t);

}  // namespace q4nx
