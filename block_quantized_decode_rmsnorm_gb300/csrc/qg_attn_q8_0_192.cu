// Decode attention over a Q8_0 cache, heads of 192 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(false, 192)
}  // namespace qg
