// q4nx_attention_own.cu -- the kernel for few query rows, a request's own positions.
#include "q4nx_attention_rows.cuh"

namespace q4nx {

template cudaError_t launch_attention_rows<kOwn>(int, bool, const AttnArgsOf<kOwn>&, int, const DeviceInfo&, cudaStream_t);

}  // namespace q4nx
