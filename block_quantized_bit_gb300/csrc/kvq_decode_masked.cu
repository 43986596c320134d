// kvq_decode_masked.cu -- the CUDA-core decode of drafted tokens (kvq_tree), each a sequence with a mask of its own.
#include "kvq_decode_cc.cuh"

namespace kvq {

kvq_status launch_decode_cc_masked(const DecodeArgs& a, cudaStream_t stream) { return launch_cc_shape<true>(a, stream); }

}  // namespace kvq
