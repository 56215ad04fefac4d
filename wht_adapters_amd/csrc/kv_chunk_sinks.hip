// Instances of the chunk kernel for a window beside a few first keys (sinks).
#include "kv_chunk.hpp"

namespace whtq {

template <int D, int T, bool INT4>
static hipError_t sinks_launch(const KvAttnArgs& a, int waves, hipStream_t s) { return chunk_launch<D, T, INT4, true>(a, waves, s); }
hipError_t launch_kv_chunk_sinks(const KvAttnArgs& a, int dim, int dt, bool int4, int waves, hipStream_t s) {
  return KV_PICK(sinks_launch, dim, dt, int4, a, waves, s);
}

}  // namespace whtq
