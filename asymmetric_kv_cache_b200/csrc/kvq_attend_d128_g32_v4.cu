// Instantiations of the attend kernels for head_dim 128, group 32, 4-bit
// values (2- and 4-bit keys).
#include "kvq_attend_tc.cuh"

namespace kvq {
KVQ_ATTEND_DEFINE(128, 4, 4, 32)
KVQ_ATTEND_DEFINE(128, 2, 4, 32)
}  // namespace kvq
