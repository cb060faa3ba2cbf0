// q4nx_attention_block_own.cu -- the kernel for many query rows, a request's own positions.
#include "q4nx_attention_block.cuh"

namespace q4nx {

template cudaError_t launch_attention_block<kOwn>(int, const AttnArgsOf<kOwn>&, int64_t, int, int, const DeviceInfo&, cudaStream_t);

}  // namespace q4nx
