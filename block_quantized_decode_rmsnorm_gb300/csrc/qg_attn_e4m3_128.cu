// Decode attention over a e4m3 cache, heads of 128 values.
#include "qg_attn.cuh"

namespace qg {
QG_ATTN_DIM(true, 128)
}  // namespace qg
