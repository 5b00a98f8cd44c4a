// Decode attention over a e4m3 cache, heads of 96 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(true, 96)
}  // namespace qg
