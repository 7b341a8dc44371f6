// k_kv_cache.cu -- the paged cache written and read back.
//
// Write: a row is one token of one kv head, D values.  For an e4m3 cache the
// row's scale is the smallest power of two 2^e with max|x| <= 448 * 2^e, taken
// from the bits of the largest magnitude (448 = 1.75 * 2^8), and the codes are
// x * 2^-e rounded to nearest even: the product is exact, so a code differs
// from the value by one rounding.  Read: code * 2^e, exact in bf16 and fp32.
//
// Both are copies: bound by memory for prompts and histories, by latency for
// one token per sequence.  D / 8 lanes take a row, 16 bytes of bf16 each, and
// a group does the K and V rows of two (token, head) pairs together, so that
// four loads per lane are in flight before the first is used; the new rows'
// places come from the index alone, and the table is read while they are on
// their way.  8 prompts of up to 4096 tokens, 8 kv heads of 128, bf16 to e4m3:
// 29.4 us, 5.1 TB/s, 76% of a copy's rate (two rows at a time in flight, the
// maxima on packed 16-bit pairs; one row at a time took 53).  Read back, 2 x
// 16384 tokens of 16 heads: 69.7 us, 84%.
#include <cuda_fp16.h>

#include "ra_paged.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256, kUnroll = 2;

// Eight consecutive values in registers.
struct Eight {
    float x[8];
};

// The same as loaded: fewer registers while they wait.
template <typename T>
struct Raw {
    uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw<T> load8(const T *p)
{
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}

__device__ __forceinline__ Eight widen(const Raw<__nv_bfloat16> &w)
{
    const uint32_t a[4] = {w.w[0].x, w.w[0].y, w.w[0].z, w.w[0].w};
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.x[2 * i] = __uint_as_float(a[i] << 16);
        r.x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
    return r;
}

__device__ __forceinline__ Eight widen(const Raw<float> &w)
{
    const uint32_t a[8] = {w.w[0].x, w.w[0].y, w.w[0].z, w.w[0].w, w.w[1].x, w.w[1].y, w.w[1].z, w.w[1].w};
    Eight r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.x[i] = __uint_as_float(a[i]);
    return r;
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Eight &r)
{
    uint4 w;
    w.x = pack_bf16x2(r.x[0], r.x[1]);
    w.y = pack_bf16x2(r.x[2], r.x[3]);
    w.z = pack_bf16x2(r.x[4], r.x[5]);
    w.w = pack_bf16x2(r.x[6], r.x[7]);
    *reinterpret_cast<uint4 *>(p) = w;
}

__device__ __forceinline__ void store8(float *p, const Eight &r)
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(r.x[0], r.x[1], r.x[2], r.x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(r.x[4], r.x[5], r.x[6], r.x[7]);
}

// codes of four values, the first in the lowest byte
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// The scale byte of a row from the bits of its largest magnitude: frexp's
// exponent less 9, or less 8 above 1.75 * 2^n; 255 when it is not finite.
__device__ __forceinline__ uint32_t row_exp(uint32_t amax_bits)
{
    if (amax_bits >= 0x7f800000u) return 255u;
    const int e = (int)(amax_bits >> 23) - 135 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(max(e, -110) + 127);
}

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

// Stores a lane's eight values of a row; 8-bit: as codes at the scale that the
// row's largest magnitude asks for.
template <int LANES, bool FP8>
__device__ __forceinline__ void put_row(const Eight &r, uint32_t top, const void *base, const uint8_t *exps, size_t row, int lane)
{
    if (FP8) {
        const uint32_t e = row_exp(top);
        // 2^-(e - 127): its exponent field is 254 - e, in [7, 237]
        const float inv = __uint_as_float((254u - e) << 23);
        uint2 w = make_uint2(0, 0);
        if (e != 255u) {
            w.x = e4m3x4(r.x[0] * inv, r.x[1] * inv, r.x[2] * inv, r.x[3] * inv);
            w.y = e4m3x4(r.x[4] * inv, r.x[5] * inv, r.x[6] * inv, r.x[7] * inv);
        }
        reinterpret_cast<uint2 *>(const_cast<uint8_t *>(static_cast<const uint8_t *>(base)) + row * (LANES * 8))[lane] = w;
        if (lane == 0) const_cast<uint8_t *>(exps)[row] = (uint8_t)e;
    } else {
        store8(static_cast<__nv_bfloat16 *>(const_cast<void *>(base)) + row * (LANES * 8) + lane * 8, r);
    }
}

// Blocks of kUnroll rows per group lie along x over one sequence's rows
// (token, head), sequences along y.
template <int D, bool FP8, typename T>
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
            const uint2 top = FP8 ? row_tops<LANES>(kr[u], vr[u]) : make_uint2(0, 0);
            if (!put[u]) continue;
            put_row<LANES, FP8>(widen(kr[u]), top.x, c.k, c.k_exp, row[u], lane);
            put_row<LANES, FP8>(widen(vr[u]), top.y, c.v, c.v_exp, row[u], lane);
        }
    }
}

// Eight values of a cached row as the cache has them, and its scale byte.
template <bool FP8>
struct Cached {
    uint4 w; // codes: .x and .y
    uint32_t e;
};

template <int D, bool FP8>
__device__ __forceinline__ Cached<FP8> get_row(const void *base, const uint8_t *exps, size_t row, int lane)
{
    Cached<FP8> r{};
    if (FP8) {
        const uint2 w = reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(base) + row * D)[lane];
        r.w.x = w.x;
        r.w.y = w.y;
        r.e = exps[row];
    } else {
        r.w = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + row * D)[lane];
    }
    return r;
}

template <bool FP8>
__device__ __forceinline__ Eight widen(const Cached<FP8> &c)
{
    if (!FP8) return widen(Raw<__nv_bfloat16>{{c.w}});
    const float s = exp_byte_scale(c.e);
    const uint32_t h[4] = {c.w.x & 0xffffu, c.w.x >> 16, c.w.y & 0xffffu, c.w.y >> 16};
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = e4m3x2_to_f16x2(h[i]);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
        r.x[2 * i] = f.x * s;
        r.x[2 * i + 1] = f.y * s;
    }
    return r;
}

template <int D, bool FP8, typename T>
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
        Cached<FP8> kr[kUnroll] = {}, vr[kUnroll] = {};
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const unsigned r = r0 + u * GROUPS, j = r / c.Hkv, h = r - j * c.Hkv;
            if (r < rows && (int)j < len) {
                if (page[u] >= 0 && page[u] < c.n_pages) {
                    const size_t row = (((size_t)page[u] * c.Hkv + h) << c.page_shift) + (j & (c.page - 1));
                    kr[u] = get_row<D, FP8>(c.k, c.k_exp, row, lane);
                    vr[u] = get_row<D, FP8>(c.v, c.v_exp, row, lane);
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
                store8(k + at, widen(kr[u]));
                store8(v + at, widen(vr[u]));
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
        if (cache_dtype == RA_E4M3)
            return c.D == 64 ? go(kv_write_kernel<64, true, T>, kp, vp) : go(kv_write_kernel<128, true, T>, kp, vp);
        return c.D == 64 ? go(kv_write_kernel<64, false, T>, kp, vp) : go(kv_write_kernel<128, false, T>, kp, vp);
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
        if (cache_dtype == RA_E4M3)
            return c.D == 64 ? go(kv_read_kernel<64, true, T>, kp, vp) : go(kv_read_kernel<128, true, T>, kp, vp);
        return c.D == 64 ? go(kv_read_kernel<64, false, T>, kp, vp) : go(kv_read_kernel<128, false, T>, kp, vp);
    };
    if (dtype == RA_BF16) return typed(static_cast<__nv_bfloat16 *>(k), static_cast<__nv_bfloat16 *>(v));
    return typed(static_cast<float *>(k), static_cast<float *>(v));
}

} // namespace ra
