// Decode attention over a q8_0 cache: heads of 64, 96 and 128 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(false, 64)
QG_ATTN_DIM(false, 96)
QG_ATTN_DIM(false, 128)
}  // namespace qg
