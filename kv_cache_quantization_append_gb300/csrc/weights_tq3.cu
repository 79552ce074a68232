// Attention weights over KVQ_TQ3_QJL keys (a translation unit per key format, compiled in parallel).
#include "weights_kernel.cuh"

namespace kvq {

size_t weights_scratch_tq3(const MultiArgs& a, int sms) {
  weights::Plan p;
  return weights::make_plan<KVQ_TQ3_QJL>(a, sms, 0, &p);
}
cudaError_t launch_weights_tq3(const MultiArgs& a, int sms, cudaStream_t s) { return weights::launch<KVQ_TQ3_QJL>(a, sms, s); }

}  // namespace kvq
