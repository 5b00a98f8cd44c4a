// The paged, block-quantized key-value cache: what its kernels share.
//
// Planes codes[page][head][token in page][dim] and scales[page][head][token in page][B]:
// the tokens of one page and head are one piece of memory, so the attention, which walks
// over the tokens of one head, copies whole pieces, and a token's row of codes never
// leaves a page.  Scales lie apart from the codes so that both keep 16-byte pieces
// (16 tokens of scales are 32 B or 64 B bytes: page sizes are multiples of 16).
#pragma once

#include "qg_e4m3.cuh"

namespace qg {

constexpr int KV_TILE = 16;  // tokens: the unit of page sizes and of the attention's copies

__host__ __device__ constexpr int kv_blocks(bool e4m3, int dim) { return e4m3 ? (dim + EB - 1) / EB : dim / QK; }

struct KvPlanes {
    uint8_t *kq, *vq;
    void *kd, *vd;  // binary16 (q8_0) or f32 (e4m3)
    int64_t n_pages;
    int page, heads, dim;
    bool e4m3;
};

}  // namespace qg
