// Decode attention over a Q8_0 cache, heads of 96 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(false, 96)
}  // namespace qg
