// Attention weights over KVQ_Q8G32 keys (a translation unit per key format, compiled in parallel).
#include "weights_kernel.cuh"

namespace kvq {

size_t weights_scratch_q8(const MultiArgs& a, int sms) { return weights::scratch_bytes<KVQ_Q8G32>(a, sms); }
cudaError_t launch_weights_q8(const MultiArgs& a, int sms, cudaStream_t s) { return weights::launch<KVQ_Q8G32>(a, sms, s); }

}  // namespace kvq
