// k_paged_f32.cu -- attention over a paged cache in fp32 arithmetic.
//
// For each query row of an item: s_j = scale <q, k_j> (capped), an online
// softmax in base 2 over the tiles of the CTA's share, and o = sum p_j v_j.
// Keys, values, logits, probabilities and sums are fp32: the cached rows are
// widened once per tile into shared memory and used by the 8 rows of an item.
// It serves fp32 queries, whose results 16-bit tensor-core operands would
// round.  Bound by the FMA pipe: 2 * 8 multiply-adds per cached value.
#include <cuda_fp16.h>
#include <math.h>

#include "ra_paged.cuh"

namespace ra {
namespace {

constexpr int kRows = kPagedF32Rows, kKeys = kPagedF32Tile, kThreads = 128;

// A tile of keys or values, fp32, rows of D + 4 floats.
template <int D, bool FP8>
__device__ __forceinline__ void fill_tile(float *dst, const void *base, const uint8_t *exps,
                                          const PagedProblem &p, const PagedPart &part, int b, int h,
                                          int t, int len)
{
    constexpr int PER = D / 8; // 8 values each
    for (int e = threadIdx.x; e < kKeys * PER; e += kThreads) {
        const int j = e / PER, x = e % PER;
        float r[8] = {};
        if (t + j < len) {
            const int page = page_entry(p, part, b, t + j);
            if (page_valid(p, page)) {
                const size_t row =
                    (((size_t)page * p.c.Hkv + h) << p.c.page_shift) + ((t + j) & (p.c.page - 1));
                if (FP8) {
                    const uint2 w =
                        reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(base) + row * D)[x];
                    const float s = exp_byte_scale(exps[row]);
                    const uint32_t c[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t y = e4m3x2_to_f16x2(c[i]);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&y));
                        r[2 * i] = f.x * s;
                        r[2 * i + 1] = f.y * s;
                    }
                } else {
                    const uint4 w = reinterpret_cast<const uint4 *>(
                        static_cast<const __nv_bfloat16 *>(base) + row * D)[x];
                    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        r[2 * i] = __uint_as_float(c[i] << 16);
                        r[2 * i + 1] = __uint_as_float(c[i] & 0xffff0000u);
                    }
                }
            }
        }
        float4 *o = reinterpret_cast<float4 *>(dst + j * (D + 4) + x * 8);
        o[0] = make_float4(r[0], r[1], r[2], r[3]);
        o[1] = make_float4(r[4], r[5], r[6], r[7]);
    }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads)
    paged_f32_kernel(PagedProblem p, PagedPart part)
{
    // o: thread t holds column t % D of rows (t / D) * OR .. + OR - 1
    constexpr int OR = kRows * D / kThreads;
    __shared__ float4 q_s4[kRows * D / 4];
    __shared__ float4 k_s4[kKeys * (D + 4) / 4], v_s4[kKeys * (D + 4) / 4];
    __shared__ float p_s[kRows][kKeys], f_s[kRows], m_s[kRows], l_s[kRows];
    float *q_s = reinterpret_cast<float *>(q_s4);
    float *k_s = reinterpret_cast<float *>(k_s4), *v_s = reinterpret_cast<float *>(v_s4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = threadIdx.x % D, row0 = threadIdx.x / D * OR;
    const float *q = static_cast<const float *>(p.q);
    begin_in_order(part);
    report_lengths(p, part);
    PagedCursor c;
    const bool any = cursor_begin(p, part, blockIdx.x, c);
    for (int n; any;) {
        n = cursor_take(c);
        const int len = part.prefix ? paged_prefix_len(p) : paged_kv_len(p, c.b);
        __syncthreads(); // the last segment's shared arrays have been read
        for (int e = threadIdx.x; e < kRows * D; e += kThreads) {
            const PagedRow r = paged_row(p, part, c, e / D);
            q_s[e] = r.limit > 0 ? q[(((size_t)r.b * p.Lq + r.i) * p.Hq + c.h * p.G + r.g) * D + e % D]
                                 : 0.f;
        }
        // warp w owns the softmax of rows 2w and 2w + 1, lane = key
        int limit[2];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[OR] = {};
#pragma unroll
        for (int u = 0; u < 2; ++u) limit[u] = paged_row(p, part, c, 2 * warp + u).limit;
        for (int t = c.t0; t < c.t0 + n; ++t) {
            __syncthreads();
            fill_tile<D, FP8>(k_s, p.c.k, p.c.k_exp, p, part, c.b, c.h, t * kKeys, len);
            fill_tile<D, FP8>(v_s, p.c.v, p.c.v_exp, p, part, c.b, c.h, t * kKeys, len);
            __syncthreads();
            float s[2] = {0.f, 0.f};
            const float4 *k4 = reinterpret_cast<const float4 *>(k_s + lane * (D + 4));
            const float4 *q4 = reinterpret_cast<const float4 *>(q_s + 2 * warp * D);
#pragma unroll 8
            for (int d = 0; d < D / 4; ++d) {
                const float4 kv = k4[d];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float4 qv = q4[u * (D / 4) + d];
                    s[u] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[u]))));
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x = s[u] * p.scale;
                if (p.soft_cap > 0.f) x = p.soft_cap * tanhf(x / p.soft_cap);
                x = t * kKeys + lane < limit[u] ? x * kLog2e : -INFINITY;
                float top = x;
#pragma unroll
                for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                const float m_new = fmaxf(m[u], top);
                const float base = m_new == -INFINITY ? 0.f : m_new;
                const float f = exp2f(m[u] - base), e = exp2f(x - base);
                float sum = e;
#pragma unroll
                for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                l[u] = l[u] * f + sum;
                m[u] = m_new;
                p_s[2 * warp + u][lane] = e;
                if (lane == 0) f_s[2 * warp + u] = f;
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < OR; ++r) o[r] *= f_s[row0 + r];
            for (int j = 0; j < kKeys; ++j) {
                const float v = v_s[j * (D + 4) + col];
#pragma unroll
                for (int r = 0; r < OR; ++r) {
                    // a value that the row does not see must not reach it,
                    // whatever it is
                    const float e = p_s[row0 + r][j];
                    if (e != 0.f) o[r] = fmaf(e, v, o[r]);
                }
            }
        }
        // a NaN logit is visible and carries itself into l and o
        if (lane == 0) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                m_s[2 * warp + u] = m[u];
                l_s[2 * warp + u] = l[u];
            }
        }
        __syncthreads();
        if (stores_whole(part, c, n)) {
            // the whole segment was here: the rows' final values
#pragma unroll
            for (int r = 0; r < OR; ++r) {
                const PagedRow x = paged_row(p, part, c, row0 + r);
                if (!x.counts) continue;
                float mr = m_s[row0 + r], lr = l_s[row0 + r], f = 1.f;
                const int hq = c.h * p.G + x.g;
                if (p.sinks) {
                    const float sink = p.sinks[hq] * kLog2e, top = fmaxf(mr, sink);
                    f = exp2f(mr - top);
                    lr = lr * f + exp2f(sink - top);
                    mr = top;
                }
                const float val = lr == 0.f ? 0.f : o[r] * f / lr;
                static_cast<float *>(p.out)[(((size_t)x.b * p.Lq + x.i) * p.Hq + hq) * D + col] = val;
                if (col == 0)
                    p.lse[((size_t)x.b * p.Hq + hq) * p.Lq + x.i] = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * kLn2;
            }
        } else {
            const size_t at = slot_row(part, c) + row0;
#pragma unroll
            for (int r = 0; r < OR; ++r)
                if (row0 + r < part.slot_rows) {
                    part.o[(at + r) * D + col] = o[r];
                    if (col == 0) {
                        part.ml[(at + r) * 2] = m_s[row0 + r];
                        part.ml[(at + r) * 2 + 1] = l_s[row0 + r];
                    }
                }
        }
        if (!cursor_next(p, part, c, n)) break;
    }
    await_previous();
}

} // namespace

cudaError_t launch_paged_f32(const PagedProblem &p, const PagedPart &part, int cache_dtype, cudaStream_t s)
{
    auto go = [&](auto kern) {
        return launch_dependent(kern, (unsigned)part.ctas, kThreads, 0, s, p, part);
    };
    if (cache_dtype == RA_E4M3) return p.c.D == 64 ? go(paged_f32_kernel<64, true>) : go(paged_f32_kernel<128, true>);
    return p.c.D == 64 ? go(paged_f32_kernel<64, false>) : go(paged_f32_kernel<128, false>);
}

} // namespace ra
