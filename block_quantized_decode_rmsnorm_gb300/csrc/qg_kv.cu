// Writing rows into the paged cache, quantized, and reading them back.
//
// Both walk over rows of 2 * heads * dim values (keys, then values) at slots that the
// caller gives.  A thread keeps its place in the row - key or value, head, block, piece
// of 8 or 16 values - and takes several rows, so that the place is computed once and a
// row costs one slot, one division by the page size and one product.
#include "qg_kv.cuh"

namespace qg {

constexpr int KT = 256;

struct KvRows {
    KvPlanes c;
    const int64_t *slots;
    int64_t rows, n_slots;
    int lanes;        // threads to a row
    int rows_at_once; // rows that a CTA takes side by side
    int shift;        // log2 of the page size, or -1
};

// Where a row lies: its page and its place in the page; false outside the cache.
__device__ __forceinline__ bool kv_place(const KvRows &a, int64_t slot, int64_t &page, int &off)
{
    if (slot < 0 || slot >= a.n_slots) return false;
    if (a.shift >= 0) {
        page = slot >> a.shift;
    } else if (slot < (int64_t(1) << 32)) {
        page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.c.page);
    } else {
        page = slot / a.c.page;
    }
    off = static_cast<int>(slot - page * a.c.page);
    return true;
}

template <typename T>
struct KvSource {
    const T *k, *v;
    int64_t k_row, k_head, v_row, v_head;
};

// Eight values of a row: two or one 16-byte loads.
template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ float4 lo() const { return a; }
    __device__ __forceinline__ float4 hi() const { return b; }
};
template <>
struct Vec8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ float4 lo() const { return Vec4<__nv_bfloat16>::widen(make_uint2(r.x, r.y)); }
    __device__ __forceinline__ float4 hi() const { return Vec4<__nv_bfloat16>::widen(make_uint2(r.z, r.w)); }
};

// Lanes that hold one scale's block, eight values each.
__host__ __device__ constexpr int write_lanes(bool e4m3, int dim) { return !e4m3 ? QK / 8 : dim == 64 ? 8 : 16; }

// The largest magnitude over the L lanes of a block (fmaxf passes over NaN).
template <int L>
__device__ __forceinline__ float block_max(float m)
{
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

template <typename T, bool E4M3, int L, int RB>
__global__ void __launch_bounds__(KT) kv_write_kernel(KvRows a, KvSource<T> s)
{
    pdl_wait();
    pdl_trigger();
    const int nb = kv_blocks(E4M3, a.c.dim), block = E4M3 ? EB : QK;
    // this thread's place in a row; U (a.lanes) and KT are multiples of L, so a block's lanes stay in one warp
    const int tid = threadIdx.x;
    const int r0 = a.rows_at_once > 1 ? tid / a.lanes : 0;
    const int j = a.rows_at_once > 1 ? tid - r0 * a.lanes : blockIdx.y * KT + tid;
    const int unit = j / L, b = unit % nb, hh = unit / nb;
    const bool value = hh >= a.c.heads;
    const int h = value ? hh - a.c.heads : hh;
    const int col = b * block + (j % L) * 8;
    const bool in_row = j < a.lanes && r0 < a.rows_at_once, live = in_row && col < a.c.dim;
    const T *src = value ? s.v + h * s.v_head + col : s.k + h * s.k_head + col;
    const int64_t stride = value ? s.v_row : s.k_row;
    uint8_t *codes = value ? a.c.vq : a.c.kq;
    void *scales = value ? a.c.vd : a.c.kd;

    Vec8<T> x[RB];
    int64_t slot[RB];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * RB * a.rows_at_once + r0;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int64_t row = first + static_cast<int64_t>(i) * a.rows_at_once;
        x[i] = Vec8<T>{};
        slot[i] = -1;
        if (live && row < a.rows) {
            slot[i] = a.slots[row];
            x[i].load(src + row * stride);
        }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const float4 lo = x[i].lo(), hi = x[i].hi();
        int64_t page;
        int off;
        const bool there = kv_place(a, slot[i], page, off);
        const int64_t at = (page * a.c.heads + h) * a.c.page + off;  // row of the planes
        uint2 w;
        if constexpr (E4M3) {
            const float m = e4m3_floor(block_max<L>(fmaxf(max_abs4(lo), max_abs4(hi))));
            const float f = __fdiv_rn(448.0f, m);
            w.x = e4m3_pack4(lo.x * f, lo.y * f, lo.z * f, lo.w * f);
            w.y = e4m3_pack4(hi.x * f, hi.y * f, hi.z * f, hi.w * f);
            if (there && j % L == 0) static_cast<float *>(scales)[at * nb + b] = __fdiv_rn(m, 448.0f);
        } else {
            float m = fmaxf(fmaxf(fmaxf(fabsf(lo.x), fabsf(lo.y)), fmaxf(fabsf(lo.z), fabsf(lo.w))),
                            fmaxf(fmaxf(fabsf(hi.x), fabsf(hi.y)), fmaxf(fabsf(hi.z), fabsf(hi.w))));
            m = block_max<L>(m);
            const float d = div127(m), rd = q8_recip(d);
            w.x = q8_pack4(lo, d, rd);
            w.y = q8_pack4(hi, d, rd);
            if (there && j % L == 0) static_cast<uint16_t *>(scales)[at * nb + b] = f2h_rn(d);
        }
        if (there) *reinterpret_cast<uint2 *>(codes + at * a.c.dim + col) = w;
    }
}

// Sixteen codes -> values -> 16 outputs.
template <typename T, bool E4M3>
__device__ __forceinline__ void kv_values(uint4 q, float d, T *out)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    float4 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (E4M3) {
            const __half2 a(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] & 0xffff), __NV_E4M3)),
                b(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> 16), __NV_E4M3));
            const float2 x = __half22float2(a), y = __half22float2(b);
            f[i] = make_float4(x.x, x.y, y.x, y.y);
        } else {
            const uint32_t u = w[i] ^ 0x80808080u;  // code + 128, placed in the mantissa of 2^23
            f[i] = make_float4(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540)) - 8388736.0f,
                               __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7541)) - 8388736.0f,
                               __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7542)) - 8388736.0f,
                               __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7543)) - 8388736.0f);
        }
        f[i] = make_float4(f[i].x * d, f[i].y * d, f[i].z * d, f[i].w * d);
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<float4 *>(out)[i] = f[i];
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint2 a = Vec4<__nv_bfloat16>::narrow(f[2 * i]), b = Vec4<__nv_bfloat16>::narrow(f[2 * i + 1]);
            reinterpret_cast<uint4 *>(out)[i] = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
}

template <typename T, bool E4M3, int RB>
__global__ void __launch_bounds__(KT) kv_read_kernel(KvRows a, T *k, T *v)
{
    pdl_wait();
    pdl_trigger();
    const int nb = kv_blocks(E4M3, a.c.dim), block = E4M3 ? EB : QK;
    const int tid = threadIdx.x;
    const int r0 = a.rows_at_once > 1 ? tid / a.lanes : 0;
    const int j = a.rows_at_once > 1 ? tid - r0 * a.lanes : blockIdx.y * KT + tid;
    if (j >= a.lanes || r0 >= a.rows_at_once) return;
    const int pieces = a.c.dim / 16, hh = j / pieces, col = (j - hh * pieces) * 16;
    const bool value = hh >= a.c.heads;
    const int h = value ? hh - a.c.heads : hh;
    const uint8_t *codes = value ? a.c.vq : a.c.kq;
    const void *scales = value ? a.c.vd : a.c.kd;
    T *dst = (value ? v : k) + h * a.c.dim + col;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * RB * a.rows_at_once + r0;
    uint4 q[RB];
    float d[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int64_t row = first + static_cast<int64_t>(i) * a.rows_at_once;
        q[i] = make_uint4(0, 0, 0, 0);
        d[i] = 0.0f;
        int64_t page;
        int off;
        if (row < a.rows && kv_place(a, a.slots[row], page, off)) {
            const int64_t at = (page * a.c.heads + h) * a.c.page + off;
            q[i] = *reinterpret_cast<const uint4 *>(codes + at * a.c.dim + col);
            const int64_t b = at * nb + col / block;
            d[i] = E4M3 ? static_cast<const float *>(scales)[b] : h2f(static_cast<const uint16_t *>(scales)[b]);
        }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int64_t row = first + static_cast<int64_t>(i) * a.rows_at_once;
        if (row < a.rows) kv_values<T, E4M3>(q[i], d[i], dst + row * a.c.heads * a.c.dim);
    }
}

namespace {

KvRows rows_args(const KvPlanes &c, const int64_t *slots, int64_t rows, int lanes)
{
    int shift = -1;
    for (int s = 4; s <= 12; ++s)
        if (c.page == 1 << s) shift = s;
    return {c, slots, rows, c.n_pages * c.page, lanes, lanes <= KT / 2 ? KT / lanes : 1, shift};
}

dim3 rows_grid(const KvRows &a, int rb)
{
    const int64_t per = static_cast<int64_t>(rb) * a.rows_at_once;
    return dim3(static_cast<unsigned>((a.rows + per - 1) / per), a.rows_at_once > 1 ? 1 : (a.lanes + KT - 1) / KT);
}

// Four rows a thread where they still give every SM eight CTAs, one where rows are few.
bool many_rows(const KvRows &a) { return a.rows * a.lanes >= int64_t(num_sms()) * 8 * 4 * KT; }

template <typename T, bool E4M3, int L>
cudaError_t write_rows(const KvRows &a, const KvSource<T> &s, cudaStream_t st)
{
    if (many_rows(a)) return launch_pdl(kv_write_kernel<T, E4M3, L, 4>, rows_grid(a, 4), dim3(KT), 0, st, a, s);
    return launch_pdl(kv_write_kernel<T, E4M3, L, 1>, rows_grid(a, 1), dim3(KT), 0, st, a, s);
}

template <typename T>
cudaError_t write_type(const KvPlanes &c, const KvSource<T> &s, const int64_t *slots, int64_t rows, cudaStream_t st)
{
    const int L = write_lanes(c.e4m3, c.dim);
    const KvRows a = rows_args(c, slots, rows, 2 * c.heads * kv_blocks(c.e4m3, c.dim) * L);
    if (!c.e4m3) return write_rows<T, false, 4>(a, s, st);
    return L == 8 ? write_rows<T, true, 8>(a, s, st) : write_rows<T, true, 16>(a, s, st);
}

template <typename T, bool E4M3>
cudaError_t read_rows(const KvRows &a, void *k, void *v, cudaStream_t st)
{
    T *kt = static_cast<T *>(k), *vt = static_cast<T *>(v);
    if (many_rows(a)) return launch_pdl(kv_read_kernel<T, E4M3, 4>, rows_grid(a, 4), dim3(KT), 0, st, a, kt, vt);
    return launch_pdl(kv_read_kernel<T, E4M3, 1>, rows_grid(a, 1), dim3(KT), 0, st, a, kt, vt);
}

}  // namespace

cudaError_t launch_kv_write(const KvPlanes &c, const void *k, int64_t k_row, int64_t k_head, const void *v,
                            int64_t v_row, int64_t v_head, int dtype, const int64_t *slots, int64_t rows,
                            cudaStream_t st)
{
    if (dtype == QG_BF16)
        return write_type<__nv_bfloat16>(c, {static_cast<const __nv_bfloat16 *>(k), static_cast<const __nv_bfloat16 *>(v),
                                             k_row, k_head, v_row, v_head}, slots, rows, st);
    return write_type<float>(c, {static_cast<const float *>(k), static_cast<const float *>(v), k_row, k_head, v_row, v_head},
                             slots, rows, st);
}

cudaError_t launch_kv_read(const KvPlanes &c, const int64_t *slots, int64_t rows, void *k, void *v, int dtype,
                           cudaStream_t st)
{
    const KvRows a = rows_args(c, slots, rows, 2 * c.heads * (c.dim / 16));
    if (dtype == QG_BF16)
        return c.e4m3 ? read_rows<__nv_bfloat16, true>(a, k, v, st) : read_rows<__nv_bfloat16, false>(a, k, v, st);
    return c.e4m3 ? read_rows<float, true>(a, k, v, st) : read_rows<float, false>(a, k, v, st);
}

}  // namespace qg
