// Attention of several queries per sequence over the cache as it stands: dispatch on the key format.  The kernels are
// in tree_kernel.cuh (trees of drafted tokens) and weights_kernel.cuh (the weight that cached positions receive).
#include "kvq_internal.cuh"

namespace kvq {

#define KVQ_FORMATS(X) X(q4) X(q8) X(tq3)
#define KVQ_DECLARE(f)                                                    \
  size_t tree_scratch_##f(const MultiArgs& a, int sms);                   \
  cudaError_t launch_tree_##f(const MultiArgs& a, int sms, cudaStream_t); \
  size_t weights_scratch_##f(const MultiArgs& a, int sms);                \
  cudaError_t launch_weights_##f(const MultiArgs& a, int sms, cudaStream_t);
KVQ_FORMATS(KVQ_DECLARE)

size_t tree_scratch_bytes(const MultiArgs& a, int sms) {
  return a.k_format == KVQ_TQ3_QJL ? tree_scratch_tq3(a, sms) : a.k_format == KVQ_Q8G32 ? tree_scratch_q8(a, sms) : tree_scratch_q4(a, sms);
}
cudaError_t launch_tree(const MultiArgs& a, int sms, cudaStream_t s) {
  return a.k_format == KVQ_TQ3_QJL ? launch_tree_tq3(a, sms, s)
         : a.k_format == KVQ_Q8G32 ? launch_tree_q8(a, sms, s)
                                   : launch_tree_q4(a, sms, s);
}
size_t weights_scratch_bytes(const MultiArgs& a, int sms) {
  return a.k_format == KVQ_TQ3_QJL   ? weights_scratch_tq3(a, sms)
         : a.k_format == KVQ_Q8G32 ? weights_scratch_q8(a, sms)
                                   : weights_scratch_q4(a, sms);
}
cudaError_t launch_weights(const MultiArgs& a, int sms, cudaStream_t s) {
  return a.k_format == KVQ_TQ3_QJL ? launch_weights_tq3(a, sms, s)
         : a.k_format == KVQ_Q8G32 ? launch_weights_q8(a, sms, s)
                                   : launch_weights_q4(a, sms, s);
}

}  // namespace kvq
