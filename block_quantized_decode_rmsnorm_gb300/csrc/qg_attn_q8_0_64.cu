// Decode attention over a Q8_0 cache, heads of 64 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(false, 64)
}  // namespace qg
