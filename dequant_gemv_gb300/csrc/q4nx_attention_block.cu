// q4nx_attention_block.cu -- the kernel for many query rows, positions up to a row's own.
#include "q4nx_attention_block.cuh"

namespace q4nx {

uint64_t attention_block_bytes(int D) { return static_cast<uint64_t>(kKvMaxCtas) * (D > 128 ? kTile : kRows) * (D + 2) * 4; }

template cudaError_t launch_attention_block<kCausal>(int, const AttnArgsOf<kCausal>&, int64_t, int, int, const DeviceInfo&, cudaStream_t);

}  // namespace q4nx
