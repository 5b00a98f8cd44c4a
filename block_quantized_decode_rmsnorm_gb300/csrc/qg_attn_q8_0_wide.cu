// Decode attention over a q8_0 cache: heads of 192 and 256 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(false, 192)
QG_ATTN_DIM(false, 256)
}  // namespace qg
