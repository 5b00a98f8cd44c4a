// Decode attention over a Q8_0 cache, heads of 256 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(false, 256)
}  // namespace qg
