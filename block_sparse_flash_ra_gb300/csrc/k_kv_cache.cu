// k_kv_cache.cu -- the paged cache written and read back.
//
// Write: a row is one token of one kv head, D values.  For an e4m3 cache the
// row's scale is the smallest power of two 2^e with max|x| <= 448 * 2^e, taken
// from the bits of the largest magnitude (448 = 1.75 * 2^8), and the codes are
// x * 2^-e rounded to nearest even: the product is exact, so a code differs
// from the value by one rounding.  For a cache in 4 bits the same holds of every
// 32 values, with max|x| <= 6 * 2^e (6 = 1.5 * 2^2) and codes of e2m1.  Read:
// code * 2^e, exact in bf16 and fp32.
//
// Both are copies: bound by memory for prompts and histories, by latency for
// one token per sequence.  D / 8 lanes take a row, 16 bytes of bf16 each, and
// a group does the K and V rows of two (token, head) pairs together, so that
// four loads per lane are in flight before the first is used; the new rows'
// places come from the index alone, and the table is read while they are on
// their way.  8 prompts of up to 4096 tokens, 8 kv heads of 128, bf16 to e4m3:
// 29.4 us, 5.1 TB/s, 76% of a copy's rate (two rows at a time in flight, the
// maxima on packed 16-bit pairs; one row at a time took 53).  Read back, 2 x
// 16384 tokens of 16 heads: 69.7 us, 84%.  4 bits, 24576 tokens of 8 heads, bf16:
// written in 31 us (63%; 72% of the issue slots), 38000 places read back in 36 (77%).
#include <type_traits>

#include "ra_rows.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256, kUnroll = 2;


// Largest magnitudes, as fp32 bits, of a K row and a V row that LANES lanes hold.
template <int LANES>
__device__ __forceinline__ uint2 row_tops(const Raw<__nv_bfloat16> &k, const Raw<__nv_bfloat16> &v)
{
    // as pairs of 16-bit integers, the two rows in one word for the shuffles
    const uint32_t m = 0x7fff7fffu;
    const uint32_t a = __vmaxu2(__vmaxu2(k.w[0].x & m, k.w[0].y & m), __vmaxu2(k.w[0].z & m, k.w[0].w & m));
    const uint32_t b = __vmaxu2(__vmaxu2(v.w[0].x & m, v.w[0].y & m), __vmaxu2(v.w[0].z & m, v.w[0].w & m));
    uint32_t t = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, o));
    return make_uint2(t << 16, t & 0xffff0000u);
}

template <int LANES>
__device__ __forceinline__ uint2 row_tops(const Raw<float> &k, const Raw<float> &v)
{
    uint2 t = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t m = 0x7fffffffu;
        t.x = max(t.x, max(max(k.w[i].x & m, k.w[i].y & m), max(k.w[i].z & m, k.w[i].w & m)));
        t.y = max(t.y, max(max(v.w[i].x & m, v.w[i].y & m), max(v.w[i].z & m, v.w[i].w & m)));
    }
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) {
        t.x = max(t.x, __shfl_xor_sync(0xffffffffu, t.x, o));
        t.y = max(t.y, __shfl_xor_sync(0xffffffffu, t.y, o));
    }
    return t;
}

// The scale byte of a row (8 bits) or of the lane's block of 32 (4 bits), by its
// largest magnitude; row_e: the bytes of the row's blocks.
template <int LANES, int CACHE>
__device__ __forceinline__ uint32_t scale_of(uint32_t top, int lane, uint32_t &row_e)
{
    if (CACHE != RA_E2M1) return row_exp(top);
    const uint32_t e = block_exp(top);
    row_e = e << (lane / 4 * 8);
#pragma unroll
    for (int o = 4; o < LANES; o <<= 1) row_e |= __shfl_xor_sync(0xffffffffu, row_e, o);
    return e;
}

// Stores a lane's eight values of a row; as codes at the scale e.
template <int LANES, int CACHE>
__device__ __forceinline__ void put_row(const Eight &r, uint32_t e, uint32_t row_e, const void *base, const uint8_t *exps, size_t row,
                                        int lane)
{
    uint8_t *bytes = static_cast<uint8_t *>(const_cast<void *>(base)), *e8 = const_cast<uint8_t *>(exps);
    if (CACHE == RA_BF16) {
        store8(static_cast<__nv_bfloat16 *>(const_cast<void *>(base)) + row * (LANES * 8) + lane * 8, r);
        return;
    }
    const float inv = exp_byte_inverse(e);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = r.x[i] * inv;
    if (CACHE == RA_E4M3) {
        uint2 w = make_uint2(0, 0);
        if (e != 255u) w = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
        reinterpret_cast<uint2 *>(bytes + row * (LANES * 8))[lane] = w;
        if (lane == 0) e8[row] = (uint8_t)e;
    } else {
        reinterpret_cast<uint32_t *>(bytes + row * (LANES * 4))[lane] = e != 255u ? e2m1x8(x) : 0u;
        if (lane == 0) {
            if (LANES == 16) reinterpret_cast<uint32_t *>(e8)[row] = row_e;
            else reinterpret_cast<uint16_t *>(e8)[row] = (uint16_t)row_e;
        }
    }
}

// Blocks of kUnroll rows per group lie along x over one sequence's rows
// (token, head), sequences along y.
template <int D, int CACHE, typename T>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(PagedCache c, const T *__restrict__ k, const T *__restrict__ v, int B, int L, size_t k_stride,
                    size_t v_stride, const int32_t *__restrict__ table, int max_pages,
                    const int32_t *__restrict__ start, const int32_t *__restrict__ count, int *status)
{
    constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
    const int lane = threadIdx.x % LANES;
    const unsigned r0 = blockIdx.x * (GROUPS * kUnroll) + threadIdx.x / LANES;
    for (int b = blockIdx.y; b < B; b += gridDim.y) {
        const int first = start[b];
        const int n = count ? min(max(count[b], 0), L) : L;
        if (blockIdx.x == 0 && threadIdx.x == 0 && count && n != count[b]) report_bad_page(status);
        const unsigned rows = (unsigned)n * c.Hkv;
        if (blockIdx.x * (unsigned)(GROUPS * kUnroll) >= rows) continue;
        Raw<T> kr[kUnroll] = {}, vr[kUnroll] = {};
        size_t row[kUnroll];
        unsigned tok[kUnroll];
        bool put[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const unsigned r = r0 + u * GROUPS;
            put[u] = r < rows;
            tok[u] = r / c.Hkv;
            const unsigned h = r - tok[u] * c.Hkv;
            if (put[u]) {
                const size_t at = (size_t)b * L + tok[u];
                kr[u] = load8(k + at * k_stride + h * D + lane * 8);
                vr[u] = load8(v + at * v_stride + h * D + lane * 8);
            }
            row[u] = h;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!put[u]) continue;
            const long long pos = (long long)first + tok[u];
            int page = -1;
            if (pos >= 0 && (pos >> c.page_shift) < max_pages)
                page = table[(size_t)b * max_pages + (pos >> c.page_shift)];
            put[u] = page >= 0 && page < c.n_pages;
            if (put[u])
                row[u] = (((size_t)page * c.Hkv + row[u]) << c.page_shift) + (size_t)(pos & (c.page - 1));
            else
                report_bad_page(status);
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint2 top = CACHE == RA_BF16 ? make_uint2(0, 0) : row_tops<CACHE == RA_E4M3 ? LANES : 4>(kr[u], vr[u]);
            uint32_t kx = 0, vx = 0;
            const uint32_t ke = scale_of<LANES, CACHE>(top.x, lane, kx), ve = scale_of<LANES, CACHE>(top.y, lane, vx);
            if (!put[u]) continue;
            put_row<LANES, CACHE>(widen(kr[u]), ke, kx, c.k, c.k_exp, row[u], lane);
            put_row<LANES, CACHE>(widen(vr[u]), ve, vx, c.v, c.v_exp, row[u], lane);
        }
    }
}

// Eight values of a cached row as the cache has them, and their scale byte.
struct Cached {
    uint4 w; // e4m3: .x and .y, e2m1: .x
    uint32_t e;
};

template <int D, int CACHE>
__device__ __forceinline__ Cached get_row(const void *base, const uint8_t *exps, size_t row, int lane)
{
    Cached r{};
    const uint8_t *bytes = static_cast<const uint8_t *>(base);
    if (CACHE == RA_BF16) {
        r.w = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + row * D)[lane];
    } else if (CACHE == RA_E4M3) {
        const uint2 w = reinterpret_cast<const uint2 *>(bytes + row * D)[lane];
        r.w.x = w.x;
        r.w.y = w.y;
        r.e = exps[row];
    } else {
        r.w.x = reinterpret_cast<const uint32_t *>(bytes + row * (D / 2))[lane];
        r.e = exps[row * (D / 32) + lane / 4];
    }
    return r;
}

template <int CACHE, typename T>
__device__ __forceinline__ void put_values(T *to, const Cached &c)
{
    if (CACHE == RA_BF16) {
        store8(to, widen(Raw<__nv_bfloat16>{{c.w}}));
        return;
    }
    const float s = exp_byte_scale(c.e);
    uint32_t h[4] = {c.w.x & 0xffffu, c.w.x >> 16, c.w.y & 0xffffu, c.w.y >> 16};
    if (CACHE == RA_E2M1) e2m1x8_to_f16(c.w.x, h);
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = CACHE == RA_E4M3 ? e4m3x2_to_f16x2(h[i]) : h[i];
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
        r.x[2 * i] = f.x * s;
        r.x[2 * i + 1] = f.y * s;
    }
    store8(to, r);
}

template <int D, int CACHE, typename T>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(PagedCache c, T *__restrict__ k, T *__restrict__ v, int B, int L, const int32_t *__restrict__ table,
                   int max_pages, const int32_t *__restrict__ kv_len, int *status)
{
    constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
    const int lane = threadIdx.x % LANES;
    const unsigned r0 = blockIdx.x * (GROUPS * kUnroll) + threadIdx.x / LANES, rows = (unsigned)L * c.Hkv;
    for (int b = blockIdx.y; b < B; b += gridDim.y) {
        const int len = kv_len[b];
        int page[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) { // beside the length, not behind it
            const int n = (int)(((r0 + u * GROUPS) / c.Hkv) >> c.page_shift);
            page[u] = n < max_pages ? table[(size_t)b * max_pages + n] : -1;
        }
        if (blockIdx.x == 0 && threadIdx.x == 0 && (len < 0 || len > L)) report_bad_page(status);
        Cached kr[kUnroll] = {}, vr[kUnroll] = {};
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const unsigned r = r0 + u * GROUPS, j = r / c.Hkv, h = r - j * c.Hkv;
            if (r < rows && (int)j < len) {
                if (page[u] >= 0 && page[u] < c.n_pages) {
                    const size_t row = (((size_t)page[u] * c.Hkv + h) << c.page_shift) + (j & (c.page - 1));
                    kr[u] = get_row<D, CACHE>(c.k, c.k_exp, row, lane);
                    vr[u] = get_row<D, CACHE>(c.v, c.v_exp, row, lane);
                } else {
                    report_bad_page(status);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const unsigned r = r0 + u * GROUPS;
            if (r < rows) {
                const size_t at = ((size_t)b * rows + r) * D + lane * 8;
                put_values<CACHE>(k + at, kr[u]);
                put_values<CACHE>(v + at, vr[u]);
            }
        }
    }
}

dim3 grid_for(int B, long long rows, int lanes)
{
    const long long per = kThreads / lanes * kUnroll;
    return dim3((unsigned)((rows + per - 1) / per), (unsigned)(B < 65535 ? B : 65535));
}

} // namespace

cudaError_t launch_kv_write(const PagedCache &c, int cache_dtype, const void *k, const void *v, int dtype,
                            int B, int L, size_t k_stride, size_t v_stride, const int32_t *page_table,
                            int max_pages, const int32_t *start, const int32_t *count, int *status,
                            cudaStream_t s)
{
    const dim3 grid = grid_for(B, (long long)L * c.Hkv, c.D / 8);
    auto go = [&](auto kern, auto *kp, auto *vp) {
        kern<<<grid, kThreads, 0, s>>>(c, kp, vp, B, L, k_stride, v_stride, page_table, max_pages, start, count,
                                       status);
        return cudaGetLastError();
    };
    auto typed = [&](auto *kp, auto *vp) {
        using T = std::remove_cv_t<std::remove_pointer_t<decltype(kp)>>;
        if (cache_dtype == RA_E2M1)
            return c.D == 64 ? go(kv_write_kernel<64, RA_E2M1, T>, kp, vp) : go(kv_write_kernel<128, RA_E2M1, T>, kp, vp);
        if (cache_dtype == RA_E4M3)
            return c.D == 64 ? go(kv_write_kernel<64, RA_E4M3, T>, kp, vp) : go(kv_write_kernel<128, RA_E4M3, T>, kp, vp);
        return c.D == 64 ? go(kv_write_kernel<64, RA_BF16, T>, kp, vp) : go(kv_write_kernel<128, RA_BF16, T>, kp, vp);
    };
    if (dtype == RA_BF16)
        return typed(static_cast<const __nv_bfloat16 *>(k), static_cast<const __nv_bfloat16 *>(v));
    return typed(static_cast<const float *>(k), static_cast<const float *>(v));
}

cudaError_t launch_kv_read(const PagedCache &c, int cache_dtype, const int32_t *page_table, int max_pages,
                           const int32_t *kv_len, int B, int L, void *k, void *v, int dtype, int *status,
                           cudaStream_t s)
{
    const dim3 grid = grid_for(B, (long long)L * c.Hkv, c.D / 8);
    auto go = [&](auto kern, auto *kp, auto *vp) {
        kern<<<grid, kThreads, 0, s>>>(c, kp, vp, B, L, page_table, max_pages, kv_len, status);
        return cudaGetLastError();
    };
    auto typed = [&](auto *kp, auto *vp) {
        using T = std::remove_pointer_t<decltype(kp)>;
        if (cache_dtype == RA_E2M1)
            return c.D == 64 ? go(kv_read_kernel<64, RA_E2M1, T>, kp, vp) : go(kv_read_kernel<128, RA_E2M1, T>, kp, vp);
        if (cache_dtype == RA_E4M3)
            return c.D == 64 ? go(kv_read_kernel<64, RA_E4M3, T>, kp, vp) : go(kv_read_kernel<128, RA_E4M3, T>, kp, vp);
        return c.D == 64 ? go(kv_read_kernel<64, RA_BF16, T>, kp, vp) : go(kv_read_kernel<128, RA_BF16, T>, kp, vp);
    };
    if (dtype == RA_BF16) return typed(static_cast<__nv_bfloat16 *>(k), static_cast<__nv_bfloat16 *>(v));
    return typed(static_cast<float *>(k), static_cast<float *>(v));
}

} // namespace ra
