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
// one token per sequence.  D / 8 lanes take a row, 16 bytes of bf16 each (half as
// many where bf16 is written in 4 bits), and a group does the K and V rows of two
// (token, head) pairs together, so that four loads per lane are in flight before
// the first is used; the new rows' places come from the index alone, and the table
// is read while they are on their way.  8 prompts of up to 4096 tokens, 8 kv heads
// of 128, bf16 to e4m3: 29.4 us, 5.1 TB/s, 76% of a copy's rate (two rows at a time
// in flight, the maxima on packed 16-bit pairs; one row at a time took 53).  Read
// back, 2 x 16384 tokens of 16 heads: 69.7 us, 84%.  4 bits, 24576 tokens of 8
// heads, bf16: written in 25.4 us (77%), 38000 places read back in 36 (77%).
#include <type_traits>

#include "ra_rows.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256, kUnroll = 2;

// Eights of a row that a lane writes: two from bf16 to 4 bits, so that half as many
// lanes find a block's scale (24576 tokens of 8 heads: 31 us with one, 25.4 with two).
// From fp32 two need 89 registers: 8 x 2048 to 4096 tokens take 50 us, with one 48.
template <typename T>
constexpr int write_eights(int cache)
{
    return cache == RA_E2M1 && sizeof(T) == 2 ? 2 : 1;
}

// Largest magnitudes, as fp32 bits, of what SHARE lanes hold of a K row and a V row.
template <int SHARE, int N>
__device__ __forceinline__ uint2 row_tops(const Raw<__nv_bfloat16> (&k)[N], const Raw<__nv_bfloat16> (&v)[N])
{
    // as pairs of 16-bit integers, the two rows in one word for the shuffles
    const uint32_t m = 0x7fff7fffu;
    uint32_t a = 0, b = 0;
#pragma unroll
    for (int y = 0; y < N; ++y) {
        const uint4 x = k[y].w[0], z = v[y].w[0];
        a = __vmaxu2(a, __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m)));
        b = __vmaxu2(b, __vmaxu2(__vmaxu2(z.x & m, z.y & m), __vmaxu2(z.z & m, z.w & m)));
    }
    uint32_t t = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
    for (int o = SHARE / 2; o; o >>= 1) t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, o));
    return make_uint2(t << 16, t & 0xffff0000u);
}

template <int SHARE, int N>
__device__ __forceinline__ uint2 row_tops(const Raw<float> (&k)[N], const Raw<float> (&v)[N])
{
    uint2 t = make_uint2(0, 0);
#pragma unroll
    for (int y = 0; y < N; ++y)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t m = 0x7fffffffu;
            const uint4 x = k[y].w[i], z = v[y].w[i];
            t.x = max(t.x, max(max(x.x & m, x.y & m), max(x.z & m, x.w & m)));
            t.y = max(t.y, max(max(z.x & m, z.y & m), max(z.z & m, z.w & m)));
        }
#pragma unroll
    for (int o = SHARE / 2; o; o >>= 1) {
        t.x = max(t.x, __shfl_xor_sync(0xffffffffu, t.x, o));
        t.y = max(t.y, __shfl_xor_sync(0xffffffffu, t.y, o));
    }
    return t;
}

// The scale byte of a row (8 bits) or of the lane's block of 32 (4 bits), by its
// largest magnitude; row_e: the bytes of the row's blocks.
template <int LANES, int SHARE, int CACHE>
__device__ __forceinline__ uint32_t scale_of(uint32_t top, int lane, uint32_t &row_e)
{
    if (CACHE != RA_E2M1) return row_exp(top);
    const uint32_t e = block_exp(top);
    row_e = e << (lane / SHARE * 8);
#pragma unroll
    for (int o = SHARE; o < LANES; o <<= 1) row_e |= __shfl_xor_sync(0xffffffffu, row_e, o);
    return e;
}

// Stores a lane's values of a row; as codes at the scale e.
template <int D, int CACHE, typename T, int N>
__device__ __forceinline__ void put_row(const Raw<T> (&r)[N], uint32_t e, uint32_t row_e, const void *base, const uint8_t *exps,
                                        size_t row, int lane)
{
    uint8_t *bytes = static_cast<uint8_t *>(const_cast<void *>(base)), *e8 = const_cast<uint8_t *>(exps);
    if (CACHE == RA_BF16) {
        store8(static_cast<__nv_bfloat16 *>(const_cast<void *>(base)) + row * D + lane * 8, widen(r[0]));
        return;
    }
    const float inv = exp_byte_inverse(e);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int y = 0; y < N; ++y) {
        const Eight v = widen(r[y]);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v.x[i] * inv;
        if (e == 255u) continue;
        if (CACHE == RA_E4M3) {
            w[0] = e4m3x4(x[0], x[1], x[2], x[3]);
            w[1] = e4m3x4(x[4], x[5], x[6], x[7]);
        } else {
            w[y] = e2m1x8(x);
        }
    }
    uint8_t *at = bytes + row * (CACHE == RA_E4M3 ? D : D / 2);
    if (CACHE == RA_E4M3 || N == 2) reinterpret_cast<uint2 *>(at)[lane] = make_uint2(w[0], w[1]);
    else reinterpret_cast<uint32_t *>(at)[lane] = w[0];
    if (lane == 0) {
        if (CACHE == RA_E4M3) e8[row] = (uint8_t)e;
        else if (D == 128) reinterpret_cast<uint32_t *>(e8)[row] = row_e;
        else reinterpret_cast<uint16_t *>(e8)[row] = (uint16_t)row_e;
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
    constexpr int N = write_eights<T>(CACHE), LANES = D / 8 / N, GROUPS = kThreads / LANES;
    constexpr int SHARE = CACHE == RA_E2M1 ? 4 / N : LANES;  // lanes that have a scale in common
    const int lane = threadIdx.x % LANES;
    const unsigned r0 = blockIdx.x * (GROUPS * kUnroll) + threadIdx.x / LANES;
    for (int b = blockIdx.y; b < B; b += gridDim.y) {
        const int first = start[b];
        const int n = count ? min(max(count[b], 0), L) : L;
        if (blockIdx.x == 0 && threadIdx.x == 0 && count && n != count[b]) report_bad_page(status);
        const unsigned rows = (unsigned)n * c.Hkv;
        if (blockIdx.x * (unsigned)(GROUPS * kUnroll) >= rows) continue;
        Raw<T> kr[kUnroll][N] = {}, vr[kUnroll][N] = {};
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
#pragma unroll
                for (int y = 0; y < N; ++y) {
                    kr[u][y] = load8(k + at * k_stride + h * D + (lane * N + y) * 8);
                    vr[u][y] = load8(v + at * v_stride + h * D + (lane * N + y) * 8);
                }
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
            const uint2 top = CACHE == RA_BF16 ? make_uint2(0, 0) : row_tops<SHARE>(kr[u], vr[u]);
            uint32_t kx = 0, vx = 0;
            const uint32_t ke = scale_of<LANES, SHARE, CACHE>(top.x, lane, kx);
            const uint32_t ve = scale_of<LANES, SHARE, CACHE>(top.y, lane, vx);
            if (!put[u]) continue;
            put_row<D, CACHE>(kr[u], ke, kx, c.k, c.k_exp, row[u], lane);
            put_row<D, CACHE>(vr[u], ve, vx, c.v, c.v_exp, row[u], lane);
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
    auto go = [&](auto kern, auto *kp, auto *vp) {
        using T = std::remove_cv_t<std::remove_pointer_t<decltype(kp)>>;
        const dim3 grid = grid_for(B, (long long)L * c.Hkv, c.D / 8 / write_eights<T>(cache_dtype));
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
