// Decode attention over a e4m3 cache, heads of 64 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(true, 64)
}  // namespace qg
