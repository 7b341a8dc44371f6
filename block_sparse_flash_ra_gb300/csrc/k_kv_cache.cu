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
// a group does its token's K row and V row together, so that two loads per
// lane are in flight before the first is used; rows are found from the flat
// index alone, and the table is read while they are on their way.
#include <cuda_fp16.h>

#include "ra_paged.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;

// Eight consecutive values in registers.
struct Eight {
    float x[8];
};

__device__ __forceinline__ Eight load8(const __nv_bfloat16 *p)
{
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.x[2 * i] = __uint_as_float(a[i] << 16);
        r.x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
    return r;
}

__device__ __forceinline__ Eight load8(const float *p)
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    return Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
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

// Quantises or rounds one row, spread over LANES lanes, into the cache.
template <int LANES, bool FP8>
__device__ __forceinline__ void put_row(const Eight &r, void *base, uint8_t *exps, size_t row, int lane)
{
    if (FP8) {
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(r.x[i]) & 0x7fffffffu);
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        const uint32_t e = row_exp(a);
        if (!base) return;
        // 2^-(e - 127): its exponent field is 254 - e, in [7, 237]
        const float inv = __uint_as_float((254u - e) << 23);
        uint2 w = make_uint2(0, 0);
        if (e != 255u) {
            w.x = e4m3x4(r.x[0] * inv, r.x[1] * inv, r.x[2] * inv, r.x[3] * inv);
            w.y = e4m3x4(r.x[4] * inv, r.x[5] * inv, r.x[6] * inv, r.x[7] * inv);
        }
        reinterpret_cast<uint2 *>(static_cast<uint8_t *>(base) + row * (LANES * 8))[lane] = w;
        if (lane == 0) exps[row] = (uint8_t)e;
    } else if (base) {
        store8(static_cast<__nv_bfloat16 *>(base) + row * (LANES * 8) + lane * 8, r);
    }
}

template <int D, bool FP8, typename T>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(PagedCache c, const T *__restrict__ k, const T *__restrict__ v, int L, long long rows,
                    size_t k_stride, size_t v_stride, const int32_t *__restrict__ table, int max_pages,
                    const int32_t *__restrict__ start, const int32_t *__restrict__ count, int *status)
{
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x % LANES;
    const long long groups = (long long)gridDim.x * (kThreads / LANES);
    const long long first = (long long)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    // every group of a block makes the same number of turns: the shuffles
    // inside a row need the whole warp
    for (long long r0 = 0; r0 < rows; r0 += groups) {
        const long long r = r0 + first;
        const bool live = r < rows;
        const long long tok = live ? r / c.Hkv : 0;
        const int h = live ? (int)(r - tok * c.Hkv) : 0;
        const int b = (int)(tok / L), i = (int)(tok - (long long)b * L);
        const Eight kr = load8(k + tok * k_stride + h * D + lane * 8);
        const Eight vr = load8(v + tok * v_stride + h * D + lane * 8);
        bool put = live && i < (count ? min(count[b], L) : L);
        size_t row = 0;
        if (put) {
            const long long pos = (long long)start[b] + i;
            int page = -1;
            if (pos >= 0 && (pos >> c.page_shift) < max_pages)
                page = table[(size_t)b * max_pages + (pos >> c.page_shift)];
            put = page >= 0 && page < c.n_pages;
            if (put)
                row = (((size_t)page * c.Hkv + h) << c.page_shift) + (size_t)(pos & (c.page - 1));
            else
                atomicMax(status, RA_STATUS_BAD_PAGE);
        }
        put_row<LANES, FP8>(kr, put ? const_cast<void *>(c.k) : nullptr, const_cast<uint8_t *>(c.k_exp), row, lane);
        put_row<LANES, FP8>(vr, put ? const_cast<void *>(c.v) : nullptr, const_cast<uint8_t *>(c.v_exp), row, lane);
        if (count && lane == 0 && live && h == 0 && i == 0 && (count[b] < 0 || count[b] > L))
            atomicMax(status, RA_STATUS_BAD_PAGE);
    }
}

template <int D, bool FP8>
__device__ __forceinline__ Eight get_row(const void *base, const uint8_t *exps, size_t row, int lane)
{
    if (!FP8) return load8(static_cast<const __nv_bfloat16 *>(base) + row * D + lane * 8);
    const uint2 w = reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(base) + row * D)[lane];
    const float s = exp_byte_scale(exps[row]);
    const uint32_t h[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
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
    kv_read_kernel(PagedCache c, T *__restrict__ k, T *__restrict__ v, int L, long long rows,
                   const int32_t *__restrict__ table, int max_pages, const int32_t *__restrict__ kv_len,
                   int *status)
{
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x % LANES;
    const long long groups = (long long)gridDim.x * (kThreads / LANES);
    const long long first = (long long)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    for (long long r = first; r < rows; r += groups) {
        const long long tok = r / c.Hkv;
        const int h = (int)(r - tok * c.Hkv);
        const int b = (int)(tok / L), j = (int)(tok - (long long)b * L);
        const int len = kv_len[b];
        Eight kr{}, vr{};
        if (j < len) {
            int page = -1;
            if ((j >> c.page_shift) < max_pages) page = table[(size_t)b * max_pages + (j >> c.page_shift)];
            if (page >= 0 && page < c.n_pages) {
                const size_t row = (((size_t)page * c.Hkv + h) << c.page_shift) + (j & (c.page - 1));
                kr = get_row<D, FP8>(c.k, c.k_exp, row, lane);
                vr = get_row<D, FP8>(c.v, c.v_exp, row, lane);
            } else {
                atomicMax(status, RA_STATUS_BAD_PAGE);
            }
        }
        store8(k + r * D + lane * 8, kr);
        store8(v + r * D + lane * 8, vr);
        if (lane == 0 && h == 0 && j == 0 && (len < 0 || len > L)) atomicMax(status, RA_STATUS_BAD_PAGE);
    }
}

int grid_for(long long rows, int lanes, int num_sms)
{
    const long long per = kThreads / lanes;
    const long long need = (rows + per - 1) / per;
    const long long most = (long long)num_sms * (2048 / kThreads);
    return (int)(need < most ? need : most);
}

} // namespace

cudaError_t launch_kv_write(const PagedCache &c, int cache_dtype, const void *k, const void *v, int dtype,
                            int B, int L, size_t k_stride, size_t v_stride, const int32_t *page_table,
                            int max_pages, const int32_t *start, const int32_t *count, int *status,
                            int num_sms, cudaStream_t s)
{
    const long long rows = (long long)B * L * c.Hkv;
    const int grid = grid_for(rows, c.D / 8, num_sms);
    auto go = [&](auto kern, auto *kp, auto *vp) {
        kern<<<grid, kThreads, 0, s>>>(c, kp, vp, L, rows, k_stride, v_stride, page_table, max_pages, start,
                                       count, status);
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
                           int num_sms, cudaStream_t s)
{
    const long long rows = (long long)B * L * c.Hkv;
    const int grid = grid_for(rows, c.D / 8, num_sms);
    auto go = [&](auto kern, auto *kp, auto *vp) {
        kern<<<grid, kThreads, 0, s>>>(c, kp, vp, L, rows, page_table, max_pages, kv_len, status);
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
