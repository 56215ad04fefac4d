// Instances of the chunk kernel without sinks.
#include "kv_chunk.hpp"

namespace whtq {

hipError_t launch_kv_chunk_sinks(const KvAttnArgs& a, int dim, int dt, bool int4, int waves, hipStream_t s);

template <int D, int T, bool INT4>
static hipError_t plain_launch(const KvAttnArgs& a, int waves, hipStream_t s) { return chunk_launch<D, T, INT4, false>(a, waves, s); }
// waves: 4, or for INT4 8; 32 rows each
hipError_t launch_kv_chunk(const KvAttnArgs& a, int dim, int dt, bool int4, int waves, hipStream_t s) {
  if (a.sinks > 0) return launch_kv_chunk_sinks(a, dim, dt, int4, waves, s);
  return KV_PICK(plain_launch, dim, dt, int4, a, waves, s);
}

}  // namespace whtq
