// k_paged_f32.cu -- attention over a paged cache in fp32 arithmetic.
//
// For each query row of an item: s_j = scale <q, k_j> (capped), an online
// softmax in base 2 over the tiles of the CTA's share, and o = sum p_j v_j.
// Logits, probabilities, sums and products are fp32.  It serves fp32 queries,
// whose results 16-bit tensor-core operands would round.
//
// Bound by issue: 2 * rows multiply-adds per cached value, its widening and the
// exchanges beside them (55% of the SMs' issue and pipes; the multiply-adds
// alone would take some 30 of the 137 us below).  So nothing passes through
// shared memory on the way: D / 8
// lanes take a key, 8 values each, with q and o of all the item's rows in
// their registers; a warp takes 16 keys (part of one page) of a tile of 64.
// The lanes' partial logits are summed by halving -- each step a lane hands
// half of its rows over and keeps the other -- which leaves one row to a lane:
// 8 exchanges instead of 32 for 8 rows, and the softmax of a row and key is
// computed once, not by 16 lanes.  V is on its way while S is computed, the
// next K while the values are summed.  Multiply-adds are packed in pairs.
// 64 sequences of 2048 tokens, 8 kv heads of 128, 32 query heads: 137 us with
// an e4m3 cache (widening: 29% of memory speed), 119 us with a bf16 one (67%);
// tiles widened into shared memory took 456.  CTAs per SM for 4 rows: e4m3
// 137 us with 4, 147 with 3; bf16, with twice the bytes on their way in
// registers, 146 and 119.  With 4 bits each lane's values have a scale of their
// own, which they are multiplied by before the rest (136 us; 8 rows 222, e4m3 231).
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "ra_rows.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kWarpKeys = 16;
static_assert(kPagedF32Tile == kWarps * kWarpKeys, "a warp's keys lie in one page");

constexpr int log2_of(int x) { return x < 2 ? 0 : 1 + log2_of(x / 2); }

// Eight cached values as the cache has them.
struct Raw8 {
    uint4 w; // e4m3: .x and .y, e2m1: .x
};

template <int CACHE>
__device__ __forceinline__ Raw8 fetch8(const void *base, size_t value)
{
    Raw8 r{};
    if (CACHE == RA_E4M3) {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(base) + value);
        r.w.x = w.x;
        r.w.y = w.y;
    } else if (CACHE == RA_E2M1) {
        r.w.x = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(base) + value / 2);
    } else {
        r.w = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + value);
    }
    return r;
}

template <int CACHE>
__device__ __forceinline__ void widen8(const Raw8 &r, float2 *x)
{
    if (CACHE == RA_BF16) {
        const uint32_t c[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = make_float2(__uint_as_float(c[i] << 16), __uint_as_float(c[i] & 0xffff0000u));
        return;
    }
    uint32_t h[4] = {r.w.x & 0xffffu, r.w.x >> 16, r.w.y & 0xffffu, r.w.y >> 16};
    if (CACHE == RA_E2M1) e2m1x8_to_f16(r.w.x, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = CACHE == RA_E4M3 ? e4m3x2_to_f16x2(h[i]) : h[i];
        x[i] = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
}

template <int D, int CACHE, int R>
__global__ void __launch_bounds__(kThreads, paged_f32_per_sm(R, CACHE != RA_BF16))
    paged_f32_kernel(PagedProblem p, PagedPart part)
{
    // e4m3: a scale for the row, which its logit and its weight take; e2m1: one for
    // each 32 values, which the lanes' values take
    constexpr bool FP8 = CACHE == RA_E4M3, FP4 = CACHE == RA_E2M1;
    constexpr int LANES = D / 8, STEP = 32 / LANES, STEPS = kWarpKeys / STEP; // lanes of a key; keys at once
    constexpr int REST = log2_of(LANES) - log2_of(R); // lanes that hold the same row, as a power of two
    constexpr uint32_t ALL = 0xffffffffu;
    __shared__ float o_s[kWarps][R * D];
    __shared__ float2 ml_s[kWarps][R];
    __shared__ int without_s[FP4 ? kWarps : 1][D / 32]; // first token without a value, by block
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LANES, kg = lane / LANES;
    const int own = sub >> REST; // the row whose softmax this lane computes
    const float *q = static_cast<const float *>(p.q);
    begin_in_order(part);
    report_lengths(p, part);
    PagedCursor c;
    const bool any = cursor_begin(p, part, blockIdx.x, c);
    for (int n; any;) {
        n = cursor_take(c);
        const int len = part.prefix ? paged_prefix_len(p) : paged_kv_len(p, c.b);
        float2 qr[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const PagedRow row = paged_row(p, part, c, r);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
            if (row.limit > 0) {
                const float4 *src = reinterpret_cast<const float4 *>(
                    q + (((size_t)row.b * p.Lq + row.i) * p.Hq + c.h * p.G + row.g) * D + sub * 8);
                a = src[0];
                b = src[1];
            }
            qr[r][0] = make_float2(a.x, a.y), qr[r][1] = make_float2(a.z, a.w);
            qr[r][2] = make_float2(b.x, b.y), qr[r][3] = make_float2(b.z, b.w);
        }
        const int limit = paged_row(p, part, c, own).limit;
        float2 o[R][4] = {};
        float m = -INFINITY, l = 0.f; // m, l: of row `own`, l of this lane's keys
        int without = 0x7fffffff; // 4 bits: this lane's first token whose block of V has no value

        // the warp's keys of tile t: their first row in the cache, or -1
        auto place = [&](int t) -> long long {
            const int first = t * kPagedF32Tile + warp * kWarpKeys;
            if (first >= len) return -1;
            const int page = page_entry(p, part, c.b, first);
            if (!page_valid(p, page)) return -1;
            return (((long long)page * p.c.Hkv + c.h) << p.c.page_shift) + (first & (p.c.page - 1));
        };
        Raw8 k[STEPS], v[STEPS];
        auto fetch = [&](Raw8 *x, const void *base, long long at, int t) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int j = s * STEP + kg;
                x[s].w = make_uint4(0, 0, 0, 0);
                if (at >= 0 && t * kPagedF32Tile + warp * kWarpKeys + j < len)
                    x[s] = fetch8<CACHE>(base, (size_t)(at + j) * D + sub * 8);
            }
        };
        long long at = place(c.t0);
        fetch(k, p.c.k, at, c.t0);
        for (int t = c.t0; t < c.t0 + n; ++t) {
            const int first = t * kPagedF32Tile + warp * kWarpKeys;
            const long long next = t + 1 < c.t0 + n ? place(t + 1) : -1;
            fetch(v, p.c.v, at, t);
            uint32_t ke[STEPS], ve[STEPS];
            if (FP8 || FP4) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int j = s * STEP + kg;
                    const bool there = at >= 0 && first + j < len; // else zeros, at a scale of one
                    const long long e = FP4 ? (at + j) * (D / 32) + sub / 4 : at + j;
                    ke[s] = there ? p.c.k_exp[e] : 127u;
                    ve[s] = there ? p.c.v_exp[e] : 127u;
                    if (FP4 && ve[s] == 255u) without = min(without, first + j);
                }
            }
            // ---- logits of row `own`
            float x[STEPS], top = -INFINITY;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                float2 kf[4];
                float d[R];
                widen8<CACHE>(k[s], kf);
                if (FP4) {
                    const float e = exp_byte_scale(ke[s]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) kf[y] = fmul2(kf[y], make_float2(e, e));
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float2 z = fmul2(qr[r][0], kf[0]);
#pragma unroll
                    for (int y = 1; y < 4; ++y) z = ffma2(qr[r][y], kf[y], z);
                    d[r] = z.x + z.y;
                }
#pragma unroll
                for (int h = R / 2, w = LANES / 2; h >= 1; h >>= 1, w >>= 1) {
                    const bool up = (sub & w) != 0;
#pragma unroll
                    for (int r = 0; r < h; ++r) {
                        const float mine = up ? d[r + h] : d[r], other = up ? d[r] : d[r + h];
                        d[r] = mine + __shfl_xor_sync(ALL, other, w);
                    }
                }
#pragma unroll
                for (int w = (1 << REST) / 2; w; w >>= 1) d[0] += __shfl_xor_sync(ALL, d[0], w);
                float z = d[0] * p.scale;
                if (FP8) z *= exp_byte_scale(ke[s]);
                if (p.soft_cap > 0.f) z = p.soft_cap * tanhf(z / p.soft_cap);
                x[s] = first + s * STEP + kg < limit ? z * kLog2e : -INFINITY;
                top = fmaxf(top, x[s]);
            }
            fetch(k, p.c.k, next, t + 1);
            at = next;
            // ---- weights
#pragma unroll
            for (int w = LANES; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(ALL, top, w));
            const float m_new = fmaxf(m, top), base = finite_base(m_new);
            if (__any_sync(ALL, m_new != m)) {
                const float f = exp2f(m - base);
                l *= f;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float fr = __shfl_sync(ALL, f, r << REST);
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[r][y] = fmul2(o[r][y], make_float2(fr, fr));
                }
                m = m_new;
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const float e = exp2f(x[s] - base);
                l += e;
                // a value that the row does not see must not reach it, whatever it is
                x[s] = !FP8 ? e : e == 0.f ? 0.f : e * exp_byte_scale(ve[s]);
            }
            // ---- values
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                float2 vf[4];
                widen8<CACHE>(v[s], vf);
                if (FP4) { // (0 for a block without a value: rows that do not see its token must not, either)
                    const float e = ve[s] == 255u ? 0.f : exp_byte_scale(ve[s]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) vf[y] = fmul2(vf[y], make_float2(e, e));
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float e = __shfl_sync(ALL, x[s], kg * LANES + (r << REST));
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[r][y] = ffma2(make_float2(e, e), vf[y], o[r][y]);
                }
            }
        }
        // ---- the segment's end: key groups of a warp, then the warps
#pragma unroll
        for (int w = LANES; w < 32; w <<= 1) {
            l += __shfl_xor_sync(ALL, l, w);
            if (FP4) without = min(without, __shfl_xor_sync(ALL, without, w));
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    o[r][y].x += __shfl_xor_sync(ALL, o[r][y].x, w);
                    o[r][y].y += __shfl_xor_sync(ALL, o[r][y].y, w);
                }
        }
        if (kg == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float4 *dst = reinterpret_cast<float4 *>(o_s[warp] + r * D + sub * 8);
                dst[0] = make_float4(o[r][0].x, o[r][0].y, o[r][1].x, o[r][1].y);
                dst[1] = make_float4(o[r][2].x, o[r][2].y, o[r][3].x, o[r][3].y);
            }
            if ((sub & ((1 << REST) - 1)) == 0) ml_s[warp][own] = make_float2(m, l);
            if (FP4 && sub % 4 == 0) without_s[warp][sub / 4] = without;
        }
        __syncthreads();
        const bool final = stores_whole(part, c, n);
        const size_t slot = slot_row(part, c);
#pragma unroll 1
        for (int e = threadIdx.x; e < R * D; e += kThreads) {
            const int r = e / D, col = e % D;
            const PagedRow row = paged_row(p, part, c, r);
            if (!row.counts) continue;
            float mr = -INFINITY, lr = 0.f, val = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mr = fmaxf(mr, ml_s[w][r].x);
            const float base = finite_base(mr);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ml = ml_s[w][r];
                const float f = exp2f(ml.x - base);
                lr += ml.y * f;
                val += o_s[w][e] * f;
                if (FP4 && without_s[w][col / 32] < row.limit) val = __uint_as_float(0x7fc00000u);
            }
            if (final) {
                const int hq = c.h * p.G + row.g;
                if (p.sinks) {
                    const float sink = p.sinks[hq] * kLog2e, with = finite_base(fmaxf(mr, sink)), f = exp2f(mr - with);
                    lr = lr * f + exp2f(sink - with);
                    val *= f;
                    mr = with;
                }
                static_cast<float *>(p.out)[(((size_t)row.b * p.Lq + row.i) * p.Hq + hq) * D + col] =
                    lr == 0.f ? 0.f : val / lr;
                if (col == 0)
                    p.lse[((size_t)row.b * p.Hq + hq) * p.Lq + row.i] = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * kLn2;
            } else {
                part.o[(slot + r) * D + col] = val;
                if (col == 0) *reinterpret_cast<float2 *>(part.ml + (slot + r) * 2) = make_float2(mr, lr);
            }
        }
        if (!cursor_next(p, part, c, n)) break;
        __syncthreads(); // o_s and ml_s are free again
    }
    await_previous();
}

} // namespace

cudaError_t launch_paged_f32(const PagedProblem &p, const PagedPart &part, int cache_dtype, cudaStream_t s)
{
    auto go = [&](auto kern) { return launch_dependent(kern, (unsigned)part.ctas, kThreads, 0, s, p, part); };
    auto sized = [&](auto d, auto cache) {
        constexpr int D = decltype(d)::value, CACHE = decltype(cache)::value;
        return part.row_block == 4 ? go(paged_f32_kernel<D, CACHE, 4>) : go(paged_f32_kernel<D, CACHE, 8>);
    };
    auto typed = [&](auto cache) {
        return p.c.D == 64 ? sized(std::integral_constant<int, 64>{}, cache) : sized(std::integral_constant<int, 128>{}, cache);
    };
    return cache_dtype == RA_E2M1   ? typed(std::integral_constant<int, RA_E2M1>{})
           : cache_dtype == RA_E4M3 ? typed(std::integral_constant<int, RA_E4M3>{})
                                    : typed(std::integral_constant<int, RA_BF16>{});
}

} // namespace ra
