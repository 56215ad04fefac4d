// Instances of the step kernel for a window beside a few first keys (sinks).
#include "kv_step.hpp"

namespace whtq {

template <int D, int T, bool INT4>
static hipError_t sinks_launch(const KvAttnArgs& a, int nq, hipStream_t s) { return step_launch<D, T, INT4, true>(a, nq, s); }
hipError_t launch_kv_step_sinks(const KvAttnArgs& a, int dim, int dt, bool int4, int nq, hipStream_t s) {
  return KV_PICK(sinks_launch, dim, dt, int4, a, nq, s);
}

}  // namespace whtq
