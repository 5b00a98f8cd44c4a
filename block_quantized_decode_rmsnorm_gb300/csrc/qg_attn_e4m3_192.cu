// Decode attention over a e4m3 cache, heads of 192 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(true, 192)
}  // namespace qg
