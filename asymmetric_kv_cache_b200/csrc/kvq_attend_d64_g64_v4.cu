// Instantiations of the attend kernels for head_dim 64, group 64, 4-bit
// values (2- and 4-bit keys).
#include "kvq_attend_tc.cuh"

namespace kvq {
KVQ_ATTEND_DEFINE(64, 4, 4, 64)
KVQ_ATTEND_DEFINE(64, 2, 4, 64)
}  // namespace kvq
