// Tree attention over KVQ_Q4G32 keys (a translation unit per key format, compiled in parallel).
#include "tree_kernel.cuh"

namespace kvq {

size_t tree_scratch_q4(const MultiArgs& a, int sms) {
  tree::Plan p;
  return tree::make_plan<KVQ_Q4G32>(a, sms, &p);
}
cudaError_t launch_tree_q4(const MultiArgs& a, int sms, cudaStream_t s) {
  return a.in_bf16 ? tree::launch<KVQ_Q4G32, false>(a, sms, s) : tree::launch<KVQ_Q4G32, true>(a, sms, s);
}

}  // namespace kvq
