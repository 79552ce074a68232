// Attention weights over KVQ_TQ3_QJL keys (a translation unit per key format, compiled in parallel).
#include "weights_kernel.cuh"

namespace kvq {

size_t weights_scratch_tq3(const MultiArgs& a, int sms) { return weights::scratch_bytes<KVQ_TQ3_QJL>(a, sms); }
cudaError_t launch_weights_tq3(const MultiArgs& a, int sms, cudaStream_t s) { return weights::launch<KVQ_TQ3_QJL>(a, sms, s); }

}  // namespace kvq
