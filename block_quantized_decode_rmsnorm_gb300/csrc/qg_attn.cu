// Decode attention: the workspace and the choice of kernel (qg_attn.cuh).
#include "qg_attn.cuh"

#include <cmath>

namespace qg {

namespace {

struct Sizes {
    int ctas, record, heads, unit, cost;  // CTAs per SM, floats of a record, query heads and tokens to a unit, an item's cost in units
};

template <bool E4M3, int D>
Sizes sizes_of(int64_t group)
{
    using One = AttnShape<E4M3, D, 1>;
    using Two = AttnShape<E4M3, D, 2>;
    if (group <= 8) return {One::CTAS, One::RECORD, One::HEADS, One::TOK * AT_WARPS, One::COST};
    return {Two::CTAS, Two::RECORD, Two::HEADS, Two::TOK * AT_WARPS, Two::COST};
}

template <bool E4M3>
Sizes sizes_for(int64_t dim, int64_t group)
{
    switch (dim) {
    case 64: return sizes_of<E4M3, 64>(group);
    case 96: return sizes_of<E4M3, 96>(group);
    case 128: return sizes_of<E4M3, 128>(group);
    case 192: return sizes_of<E4M3, 192>(group);
    default: return sizes_of<E4M3, 256>(group);
    }
}

int64_t counter_bytes() { return (static_cast<int64_t>(num_sms()) * AT_CTAS_MAX * 4 + 255) / 256 * 256; }

template <bool E4M3>
cudaError_t launch_for(const AttnArgs &a, int64_t most, cudaStream_t st)
{
    switch (a.c.dim) {
    case 64: return launch_attn_dim<E4M3, 64>(a, most, st);
    case 96: return launch_attn_dim<E4M3, 96>(a, most, st);
    case 128: return launch_attn_dim<E4M3, 128>(a, most, st);
    case 192: return launch_attn_dim<E4M3, 192>(a, most, st);
    default: return launch_attn_dim<E4M3, 256>(a, most, st);
    }
}

}  // namespace

// Counters, then two records for every CTA that the larger of the two formats' kernels has.
int64_t attn_workspace_bytes(int64_t q_heads, int64_t heads, int64_t dim)
{
    const Sizes a = sizes_for<false>(dim, q_heads / heads), b = sizes_for<true>(dim, q_heads / heads);
    const int64_t floats = a.ctas > b.ctas ? static_cast<int64_t>(a.ctas) * a.record : static_cast<int64_t>(b.ctas) * b.record;
    return counter_bytes() + num_sms() * floats * 2 * 4;
}

// The places that the line can have: by the page tables' width, or a window that may begin inside a step.
int64_t attn_most_places(const KvPlanes &c, int64_t batch, int64_t q_heads, int64_t max_pages, int64_t window)
{
    const int64_t group = q_heads / c.heads;
    const Sizes s = c.e4m3 ? sizes_for<true>(c.dim, group) : sizes_for<false>(c.dim, group);
    int64_t tokens = max_pages * c.page;
    if (window > 0 && window < tokens) tokens = window + s.unit;
    return batch * c.heads * ((group + s.heads - 1) / s.heads) * ((tokens + s.unit - 1) / s.unit + s.cost);
}

// The form of a call on `items` items of at most `tokens` tokens.  -1, the warps' form: where the items are more than find
// room at a CTA to each, and a warp has few steps to an item: AT_SHORT, or twice as many where the items are three times
// the room.  Measured from just above the room to twelve times it, for all head sizes (4 query heads of 128 to a head, Q8_0,
// the warps' time and the line's): 1024 items of 16 tokens 6.1 and 14.9 us, of 256 (8 steps) 18.1 and 28.5, of 512 (16) 31.1
// and 36.3; 305 of 256 13.7 and 13.7, of 512 22.8 and 16.4; 608 of 512 23.8 and 24.9.  Heads of 256: 305 of 256 (16 steps)
// 26.5 and 18.3, 1024 of 256 33.1 and 39.3, of 512 58.4 and 48.4.
// Otherwise the direct form's CTAs to an item, or 0 for the line: direct where each CTA has at most four units of the widest item (four units:
// 1 x 4096 tokens, 8 heads 8.3 us, 10.1 in the line; eight: 8 x 2048 tokens 12.4, 10.9 in the line), and all items are
// resident at once.  Clusters double while they are not more than half of the SMs together.
int form_of(int64_t items, int64_t most, int64_t tokens, const Sizes &s)
{
    const int64_t units = most / items - s.cost;
    int n = 1;
    while (n < AT_CLUSTER && n < units && items * n * 2 <= num_sms()) n *= 2;
    const int64_t room = static_cast<int64_t>(num_sms()) * s.ctas;
    const int64_t step = s.unit / AT_WARPS, steps = (tokens + step - 1) / step;
    if (items > room && steps <= (items < 3 * room ? AT_SHORT : 2 * AT_SHORT)) return -1;
    return items * n <= room && (units + n - 1) / n <= 4 ? n : 0;
}

cudaError_t launch_attn_decode(const KvPlanes &c, const void *q, int64_t q_row, int64_t q_head, int q_dtype,
                               int64_t batch, int64_t q_heads, const int32_t *pages, int64_t max_pages,
                               const int32_t *lengths, float scale, int64_t window, void *out, int out_dtype,
                               float *lse, void *workspace, cudaStream_t st)
{
    const int64_t group = q_heads / c.heads;
    const Sizes s = c.e4m3 ? sizes_for<true>(c.dim, group) : sizes_for<false>(c.dim, group);
    int shift = -1;
    for (int i = 4; i <= 12; ++i)
        if (c.page == 1 << i) shift = i;
    AttnArgs a = {};
    a.c = c;
    a.q = q, a.q_row = q_row, a.q_head = q_head, a.q_bf16 = q_dtype == QG_BF16;
    a.group = static_cast<int>(group), a.q_heads = static_cast<int>(q_heads);
    a.chunks = static_cast<int>((group + s.heads - 1) / s.heads);
    a.page_shift = shift;
    a.batch = batch, a.pages = pages, a.lengths = lengths, a.max_pages = max_pages;
    a.exponent = std::fabs(scale) > 0x1p126f ? 2 : 0;
    a.factor = (a.exponent ? scale * 0.25f : scale) * kLog2e;
    a.most = std::isfinite(scale) ? FLT_MAX : INFINITY;
    a.held = static_cast<int>(max_pages * c.page);
    a.window = window < a.held ? static_cast<int>(window) : 0;  // one that reaches over the whole table is none
    a.out = out, a.out_bf16 = out_dtype == QG_BF16, a.lse = lse;
    a.counters = static_cast<int *>(workspace);
    a.records = reinterpret_cast<float *>(static_cast<char *>(workspace) + counter_bytes());
    const int64_t most = attn_most_places(c, batch, q_heads, max_pages, window);
    a.narrow = most < (int64_t(1) << 31);
    a.cluster = form_of(batch * c.heads * a.chunks, most, window > 0 && window < max_pages * c.page ? window : max_pages * c.page, s);
    return c.e4m3 ? launch_for<true>(a, most, st) : launch_for<false>(a, most, st);
}

}  // namespace qg
