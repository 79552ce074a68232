// Tree attention over KVQ_TQ3_QJL keys (a translation unit per key format, compiled in parallel).
#include "tree_kernel.cuh"

namespace kvq {

size_t tree_scratch_tq3(const MultiArgs& a, int sms) {
  tree::Plan p;
  return tree::make_plan<KVQ_TQ3_QJL>(a, sms, &p);
}
cudaError_t launch_tree_tq3(const MultiArgs& a, int sms, cudaStream_t s) {
  return a.in_bf16 ? tree::launch<KVQ_TQ3_QJL, false>(a, sms, s) : tree::launch<KVQ_TQ3_QJL, true>(a, sms, s);
}

}  // namespace kvq
