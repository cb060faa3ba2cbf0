// q4nx_attention_all.cu -- the kernel for few query rows, all positions.
#include "q4nx_attention_rows.cuh"

namespace q4nx {

template cudaError_t launch_attention_rows<kAll>(int, bool, const AttnArgsOf<kAll>&, int, const DeviceInfo&, cudaStream_t);

}  // namespace q4nx
