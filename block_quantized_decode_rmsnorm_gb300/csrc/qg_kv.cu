// Writing rows into the paged cache, quantized, and reading them back.
//
// Both walk over rows of 2 * heads * dim values (keys, then values) at slots that the
// caller gives.  A thread keeps its place in the row - key or value, head, block, piece
// of 16 values - and takes several rows, so that the place is computed once and a
// row costs one slot, one division by the page size and one product.
#include <cfloat>

#include "qg_kv.cuh"

namespace qg {

constexpr int KT = 128;  // with 256: 8192 rows written 13.8 us, 13.1 with 128; 16384 read 21.5, 20.6

struct KvRows {
    KvPlanes c;
    const int64_t *slots;
    int64_t rows, n_slots;
    int lanes;        // threads to a row
    int rows_at_once; // rows that a CTA takes side by side
    int shift;        // log2 of the page size, or -1
};

// Which row of the planes' first head a slot is; false outside the cache.  Head h's is h * page_size rows on.
__device__ __forceinline__ bool kv_place(const KvRows &a, int64_t slot, int64_t &row)
{
    row = 0;
    if (slot < 0 || slot >= a.n_slots) return false;
    uint32_t page;  // fewer than 2^31
    if (a.shift >= 0) {
        page = static_cast<uint32_t>(slot >> a.shift);
    } else if (slot < (int64_t(1) << 32)) {
        page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.c.page);
    } else {
        page = static_cast<uint32_t>(slot / a.c.page);
    }
    const uint32_t size = a.c.page, off = static_cast<uint32_t>(slot) - page * size;  // mod 2^32
    row = static_cast<int64_t>(static_cast<uint64_t>(page) * (size * a.c.heads) + off);
    return true;
}

template <typename T>
struct KvSource {
    const T *k, *v;
    int64_t k_row, k_head, v_row, v_head;
};

// Sixteen values of a row.
template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
    float4 r[4];
    __device__ __forceinline__ void load(const float *p)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = reinterpret_cast<const float4 *>(p)[i];
    }
    __device__ __forceinline__ float4 get(int i) const { return r[i]; }
};
template <>
struct Vec16<__nv_bfloat16> {
    uint4 r[2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        r[0] = reinterpret_cast<const uint4 *>(p)[0];
        r[1] = reinterpret_cast<const uint4 *>(p)[1];
    }
    __device__ __forceinline__ float4 get(int i) const
    {
        const uint4 v = r[i / 2];
        return Vec4<__nv_bfloat16>::widen(i % 2 ? make_uint2(v.z, v.w) : make_uint2(v.x, v.y));
    }
};

// Lanes that hold one scale's block, sixteen values each.
__host__ __device__ constexpr int write_lanes(bool e4m3, int dim) { return !e4m3 ? QK / 16 : dim == 64 ? 4 : 8; }

// The largest magnitude over the L lanes of a block, NaN passed over, ...
template <int L>
__device__ __forceinline__ float block_max(float m)
{
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
// ... and NaN if there is one.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The Q8_0 codes of sixteen values of a block with scale d, 2^-100 <= d < infinity, none of them NaN: those of q8_code,
// without a branch (in a bf16 row 0.4 % of the values are exact halves of d, so that a branch to the division is taken by
// most warps).  The quotient is corrected once (Markstein): with y = 1 / d correctly rounded, t = fl(v y) and the exact
// r = v - t d, fl(t + r y) is the rounded quotient up to 2^-24 of an ulp; that it lies on the same side of every
// half-integer as fl(v / d) was checked for all 2^23 mantissas of d and the five floats around each of the 127 places
// where it matters (orc_corrected_quotients_off of the oracle; the tests run a part of it).  Adding 1/2 and 2^23 toward zero
// leaves the magnitude rounded half away from zero.
__device__ __forceinline__ uint4 q8_codes16(const float4 (&v)[4], float d)
{
    const float y = __frcp_rn(d);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float t = __fmul_rn(x[j], y), r = __fmaf_rn(-t, d, x[j]);
            const float q = __fmaf_rn(r, y, t);
            s[j] = __float_as_uint(__fadd_rz(__fadd_rz(fabsf(q), 0.5f), 8388608.0f));
        }
        const uint32_t p = __byte_perm(__byte_perm(s[0], s[1], 0x0040), __byte_perm(s[2], s[3], 0x0040), 0x5410);
        // bytes of negative values other than 0 to two's complement
        const uint32_t top = __byte_perm(__byte_perm(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x0073),
                                         __byte_perm(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x0073), 0x5410);
        uint32_t minus;  // 255 where top's byte has its highest bit and p's is not 0
        asm("prmt.b32 %0, %1, 0, 0xba98;" : "=r"(minus) : "r"(top & (p + 0x7f7f7f7fu)));
        w[i] = (p ^ minus) + (minus & 0x01010101u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Any block's, one value after the other.
__device__ __noinline__ uint4 q8_codes16_any(float4 a, float4 b, float4 c, float4 e, float d)
{
    const float rd = q8_recip(d);
    return make_uint4(q8_pack4(a, d, rd), q8_pack4(b, d, rd), q8_pack4(c, d, rd), q8_pack4(e, d, rd));
}

// Bound by issue where rows are many (8192 rows of 8 heads of 128 bf16 values in Q8_0: 12.8 us for 51 MB, in e4m3 10.3; 0.7
// instructions a cycle and scheduler): eight instructions a code, and the slot's, the addresses' and the maximum's beside them.
template <typename T, bool E4M3, int L, int RB>
__global__ void __launch_bounds__(KT) kv_write_kernel(KvRows a, KvSource<T> s)
{
    pdl_wait();
    pdl_trigger();
    const int nb = kv_blocks(E4M3, a.c.dim), block = E4M3 ? EB : QK;
    // this thread's place in a row; a.lanes and KT are multiples of L, so a block's lanes stay in one warp
    const int tid = threadIdx.x;
    const int r0 = a.rows_at_once > 1 ? tid / a.lanes : 0;
    const int j = a.rows_at_once > 1 ? tid - r0 * a.lanes : blockIdx.y * KT + tid;
    const int unit = j / L, hh = unit / nb, b = unit - hh * nb;
    const bool value = hh >= a.c.heads;
    const int h = value ? hh - a.c.heads : hh;
    const int col = b * block + (j % L) * 16;
    const bool live = j < a.lanes && r0 < a.rows_at_once && col < a.c.dim;
    const T *src = value ? s.v + h * s.v_head + col : s.k + h * s.k_head + col;
    const int64_t stride = value ? s.v_row : s.k_row;
    const int64_t head_row = static_cast<int64_t>(h) * a.c.page;
    uint8_t *const codes = (value ? a.c.vq : a.c.kq) + head_row * a.c.dim + col;
    const int64_t scale_at = head_row * nb + b;
    void *const scales = value ? a.c.vd : a.c.kd;

    Vec16<T> x[RB];
    int64_t slot[RB];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * RB * a.rows_at_once + r0;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int64_t row = first + static_cast<int64_t>(i) * a.rows_at_once;
        x[i] = Vec16<T>{};
        slot[i] = -1;
        if (live && row < a.rows) {
            slot[i] = a.slots[row];
            x[i].load(src + row * stride);
        }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        float4 v[4];
        float m = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] = x[i].get(q);
            if constexpr (E4M3)
                m = fmaxf(m, max_abs4(v[q]));
            else
                m = max_nan(max_nan(max_nan(m, fabsf(v[q].x)), max_nan(fabsf(v[q].y), fabsf(v[q].z))), fabsf(v[q].w));
        }
        int64_t at;
        const bool there = kv_place(a, slot[i], at);
        uint4 w;
        if constexpr (E4M3) {
            m = e4m3_floor(block_max<L>(m));
            const float f = __fdiv_rn(448.0f, m);
            w.x = e4m3_pack4(v[0].x * f, v[0].y * f, v[0].z * f, v[0].w * f);
            w.y = e4m3_pack4(v[1].x * f, v[1].y * f, v[1].z * f, v[1].w * f);
            w.z = e4m3_pack4(v[2].x * f, v[2].y * f, v[2].z * f, v[2].w * f);
            w.w = e4m3_pack4(v[3].x * f, v[3].y * f, v[3].z * f, v[3].w * f);
            if (there && j % L == 0) static_cast<float *>(scales)[at * nb + scale_at] = __fdiv_rn(m, 448.0f);
        } else {
#pragma unroll
            for (int o = L / 2; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            // a block with a NaN or an infinity has that for its scale, so that it reads as NaN: none passes for a number
            const bool odd = !(m <= FLT_MAX);
            const float d = odd ? m : div127(m);
            if (d >= 0x1p-100f && !odd)
                w = q8_codes16(v, d);
            else
                w = odd ? make_uint4(0, 0, 0, 0) : q8_codes16_any(v[0], v[1], v[2], v[3], d);
            if (there && j % L == 0) static_cast<uint16_t *>(scales)[at * nb + scale_at] = f2h_rn(d);
        }
        if (there) *reinterpret_cast<uint4 *>(codes + at * a.c.dim) = w;
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
            const uint2 p = Vec4<__nv_bfloat16>::narrow(f[2 * i]), r = Vec4<__nv_bfloat16>::narrow(f[2 * i + 1]);
            reinterpret_cast<uint4 *>(out)[i] = make_uint4(p.x, p.y, r.x, r.y);
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
    const int64_t head_row = static_cast<int64_t>(h) * a.c.page, scale_at = head_row * nb + col / block;
    const uint8_t *const codes = (value ? a.c.vq : a.c.kq) + head_row * a.c.dim + col;
    const void *const scales = value ? a.c.vd : a.c.kd;
    T *dst = (value ? v : k) + h * a.c.dim + col;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * RB * a.rows_at_once + r0;
    uint4 q[RB];
    float d[RB];
    int64_t slot[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int64_t row = first + static_cast<int64_t>(i) * a.rows_at_once;
        slot[i] = row < a.rows ? a.slots[row] : -1;
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        q[i] = make_uint4(0, 0, 0, 0);
        d[i] = 0.0f;
        int64_t at;
        if (kv_place(a, slot[i], at)) {
            q[i] = *reinterpret_cast<const uint4 *>(codes + at * a.c.dim);
            const int64_t b = at * nb + scale_at;
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

// Rows a thread: two where they still give every SM twelve CTAs (with CTAs of 256: 8192 rows written: 15.1 us with one, 13.7 with two, 13.9 with
// four; 16384 read: 23.0, 21.3, 23.3), one where rows are few.
constexpr int KRB = 2;
bool many_rows(const KvRows &a) { return a.rows * a.lanes >= int64_t(num_sms()) * 12 * KRB * KT; }

template <typename T, bool E4M3, int L>
cudaError_t write_rows(const KvRows &a, const KvSource<T> &s, cudaStream_t st)
{
    if (many_rows(a)) return launch_pdl(kv_write_kernel<T, E4M3, L, KRB>, rows_grid(a, KRB), dim3(KT), 0, st, a, s);
    return launch_pdl(kv_write_kernel<T, E4M3, L, 1>, rows_grid(a, 1), dim3(KT), 0, st, a, s);
}

template <typename T>
cudaError_t write_type(const KvPlanes &c, const KvSource<T> &s, const int64_t *slots, int64_t rows, cudaStream_t st)
{
    const int L = write_lanes(c.e4m3, c.dim);
    const KvRows a = rows_args(c, slots, rows, 2 * c.heads * kv_blocks(c.e4m3, c.dim) * L);
    if (!c.e4m3) return write_rows<T, false, 2>(a, s, st);
    return L == 4 ? write_rows<T, true, 4>(a, s, st) : write_rows<T, true, 8>(a, s, st);
}

template <typename T, bool E4M3>
cudaError_t read_rows(const KvRows &a, void *k, void *v, cudaStream_t st)
{
    T *kt = static_cast<T *>(k), *vt = static_cast<T *>(v);
    if (many_rows(a)) return launch_pdl(kv_read_kernel<T, E4M3, KRB>, rows_grid(a, KRB), dim3(KT), 0, st, a, kt, vt);
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
