// Decode attention over a e4m3 cache: heads of 64, 96 and 128 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(true, 64)
QG_ATTN_DIM(true, 96)
QG_ATTN_DIM(true, 128)
}  // namespace qg
