// k_qk.cu -- RMS norms of each head's queries and keys and their rotation by
// position, in one pass: forward, backward, and on the way into a paged cache.
//
//   z = x r, r = (mean x^2 + eps)^-1/2;  u = z w;  y = amplitude R(angle) u
// where R turns pairs of the first `rot` of a head's D values, and
//   g = amplitude R^T dy;  dw = sum g z;  dx = r (a - z mean(a z)), a = g w.
// Everything is fp32 and rounded once, to the output's type.
//
// Angles.  A pair's frequency is a number of turns per position, kept as a
// fraction of 2^64: position times frequency modulo 2^64 is the angle's
// fraction of a turn, exactly, for any 32-bit position and either sign; its
// upper 32 bits go to sincospi.  (An angle in fp32 would be off by 2^-24 of
// itself, 0.008 of a radian at position 131072.)
//
// Bound by memory: a value is read and written once and costs some ten
// operations.  A row's D values lie in D / 16 lanes, 16 values each, so that a
// warp has 4 (D = 64: 8) rows and a norm's sum is 3 (2) exchanges; with pairs
// half of `rot` apart a lane takes the eight values l and the eight that they
// are paired with, otherwise 16 in a row, so that no pair is split.  A CTA takes
// a few tokens at a time: their cosines and sines go to shared memory once, for
// all heads; then each warp takes units of two rows per lane group, all of one
// kind (queries, keys, values), whose loads are issued together.
#include <type_traits>

#include "ra_qk.h"
#include "ra_rows.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kUnroll = 2;
constexpr uint32_t kAll = 0xffffffffu;

// Cosines and sines of a step's tokens: [token][j][lane of a row] of two pairs,
// so that the lanes of a row read neighbouring words.
struct Turns {
    float4 t[kQkTokens][4][8];
};

// Lane l's 16 values of a row are the eights c0 and c1 of it.
struct Place {
    int c0, c1;
    bool turned;
};

template <bool HALF>
__device__ __forceinline__ Place place_of(int l, int rot)
{
    const bool turned = l * 16 < rot;
    if (HALF && turned) return {l, l + rot / 16, true};
    return {2 * l, 2 * l + 1, turned};
}

template <typename T>
struct Raw16 {
    Raw<T> a, b;
};

template <typename T>
__device__ __forceinline__ Raw16<T> load16(const T *row, const Place &at)
{
    return {load8(row + at.c0 * 8), load8(row + at.c1 * 8)};
}

template <typename T>
__device__ __forceinline__ void widen16(const Raw16<T> &r, float *x)
{
    const Eight a = widen(r.a), b = widen(r.b);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = a.x[i], x[8 + i] = b.x[i];
}

template <typename T>
__device__ __forceinline__ void store16(T *row, const Place &at, const float *x)
{
    Eight a, b;
#pragma unroll
    for (int i = 0; i < 8; ++i) a.x[i] = x[i], b.x[i] = x[8 + i];
    store8(row + at.c0 * 8, a);
    store8(row + at.c1 * 8, b);
}

// The sum over the lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

// Turns a lane's eight pairs by the token's angles (back: the other way).
template <bool HALF>
__device__ __forceinline__ void turn16(float *x, const float4 (*t)[8], int l, bool back)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 cs = t[j][l]; // of pairs 8 l + 2 j and the next
        const float s0 = back ? -cs.y : cs.y, s1 = back ? -cs.w : cs.w;
        const int i0 = HALF ? 2 * j : 4 * j, p0 = HALF ? 8 + 2 * j : 4 * j + 1;
        const int i1 = HALF ? 2 * j + 1 : 4 * j + 2, p1 = HALF ? 9 + 2 * j : 4 * j + 3;
        const float a0 = x[i0], b0 = x[p0], a1 = x[i1], b1 = x[p1];
        x[i0] = a0 * cs.x - b0 * s0;
        x[p0] = b0 * cs.x + a0 * s0;
        x[i1] = a1 * cs.z - b1 * s1;
        x[p1] = b1 * cs.z + a1 * s1;
    }
}

__device__ __forceinline__ long long position_of(const QkProblem &p, long long token)
{
    if (p.pos) return p.pos[token];
    const long long b = token / p.L;
    return token - b * p.L + (p.start ? p.start[b] : 0) + (p.prefix_len ? *p.prefix_len : 0);
}

// Fills the table for tokens [first, first + n).
__device__ __forceinline__ void fill_turns(Turns &turns, const QkProblem &p, long long first, int n)
{
    const int pairs = p.rot / 2;
    for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
        const int t = i / pairs, pair = i - t * pairs;
        const uint64_t turn = (uint64_t)position_of(p, first + t) * p.freq[pair];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
        float2 *to = reinterpret_cast<float2 *>(&turns.t[t][(pair & 7) >> 1][pair >> 3]) + (pair & 1);
        *to = make_float2(c * p.amplitude, s * p.amplitude);
    }
}

// A lane's 16 weights of a norm.
__device__ __forceinline__ void load_weights(float *w, const void *from, int dtype, const Place &at)
{
    if (!from) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = 1.f;
    } else if (dtype == RA_BF16) {
        widen16(load16(static_cast<const __nv_bfloat16 *>(from), at), w);
    } else {
        widen16(load16(static_cast<const float *>(from), at), w);
    }
}

// Largest magnitude of eight values, as fp32 bits.
__device__ __forceinline__ uint32_t top8(const float *x)
{
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(x[i]) & 0x7fffffffu);
    return t;
}

// Stores rows of the cache, one per group of LANES lanes (`put`: there is one),
// each lane the eights c0 and c1.  tops: 32 words of the warp.
template <int D>
__device__ __forceinline__ void put_rows(const float *x, const Place &at, bool put, const void *base, const uint8_t *exps,
                                         int dtype, size_t row, uint32_t *tops)
{
    constexpr int LANES = D / 16;
    uint8_t *bytes = static_cast<uint8_t *>(const_cast<void *>(base)), *e8 = const_cast<uint8_t *>(exps);
    if (dtype == RA_BF16) {
        if (put) store16(reinterpret_cast<__nv_bfloat16 *>(bytes) + row * D, at, x);
        return;
    }
    const int lane = threadIdx.x & 31, l = lane % LANES;
    uint32_t t0 = top8(x), t1 = top8(x + 8);
    if (dtype == RA_E4M3) {
        t0 = max(t0, t1);
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) t0 = max(t0, __shfl_xor_sync(kAll, t0, o));
        t1 = t0;
    } else {
        // a block is four eights, whichever lanes have them
        uint32_t *mine = tops + (lane / LANES) * (D / 8);
        __syncwarp();
        mine[at.c0] = t0;
        mine[at.c1] = t1;
        __syncwarp();
        const uint4 a = reinterpret_cast<const uint4 *>(mine)[at.c0 >> 2], b = reinterpret_cast<const uint4 *>(mine)[at.c1 >> 2];
        t0 = max(max(a.x, a.y), max(a.z, a.w));
        t1 = max(max(b.x, b.y), max(b.z, b.w));
    }
    if (!put) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = h ? at.c1 : at.c0;
        const uint32_t e = dtype == RA_E4M3 ? row_exp(h ? t1 : t0) : block_exp(h ? t1 : t0);
        const float inv = exp_byte_inverse(e);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[8 * h + i] * inv;
        if (dtype == RA_E4M3) {
            uint2 w = make_uint2(0, 0);
            if (e != 255u) w = make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
            *reinterpret_cast<uint2 *>(bytes + row * D + c * 8) = w;
            if (h == 0 && l == 0) e8[row] = (uint8_t)e;
        } else {
            *reinterpret_cast<uint32_t *>(bytes + row * (D / 2) + c * 4) = e != 255u ? e2m1x8(y) : 0u;
            if (c % 4 == 0) e8[row * (D / 32) + c / 4] = (uint8_t)e;
        }
    }
}

// Units of one kind: rows [0, heads) in steps of a unit's, U per lane group.
template <int LANES, int U = kUnroll>
constexpr int kUnitRows = 32 / LANES * U;
template <int LANES, int U = kUnroll>
__host__ __device__ __forceinline__ int units_of(int heads)
{
    return (heads + kUnitRows<LANES, U> - 1) / kUnitRows<LANES, U>;
}

// What the forward does with its rows: they go out, or into a cache.
struct NoCache {
};

template <int D, bool HALF, bool NORM, typename T, class TO>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && !(NORM && std::is_same<TO, QkEnter>::value) ? 4 : 3)
    qk_forward_kernel(QkProblem p, QkRows q, QkRows k, QkRows v, QkRows q_out, QkRows k_out, TO to, int step)
{
    constexpr bool ENTER = std::is_same<TO, QkEnter>::value;
    constexpr int LANES = D / 16, GROUPS = 32 / LANES;
    __shared__ Turns turns;
    __shared__ long long at_row[kQkTokens]; // ENTER: the token's first row in the cache, -1: in none, -2: left out
    __shared__ __align__(16) uint32_t tops[kWarps][32 / LANES * (D / 8)];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, group = lane / LANES;
    const long long first = (long long)blockIdx.x * step;
    const int n = (int)min((long long)step, (long long)p.B * p.L - first);
    fill_turns(turns, p, first, n);
    if constexpr (ENTER) {
        if ((int)threadIdx.x < n) {
            const long long token = first + threadIdx.x, b = token / p.L;
            const int i = (int)(token - b * p.L);
            long long row = -2;
            const int kept = to.count ? min(max(to.count[b], 0), p.L) : p.L;
            if (i == 0 && to.count && kept != to.count[b]) report_bad_page(to.status);
            if (i < kept) {
                const long long pos = (long long)p.start[b] + i;
                int page = -1;
                if (pos >= 0 && (pos >> to.c.page_shift) < to.max_pages)
                    page = to.table[(size_t)b * to.max_pages + (pos >> to.c.page_shift)];
                row = -1;
                if (page >= 0 && page < to.c.n_pages)
                    row = (((long long)page * p.Hkv) << to.c.page_shift) + (pos & (to.c.page - 1));
                else
                    report_bad_page(to.status);
            }
            at_row[threadIdx.x] = row;
        }
    }
    __syncthreads();
    const int uq = units_of<LANES>(p.Hq), uk = units_of<LANES>(p.Hkv), units = uq + uk + (ENTER ? uk : 0);
    const bool back = p.inverse != 0;
#pragma unroll 1
    for (int u = warp; u < n * units; u += kWarps) {
        const int t = u / units, in = u - t * units;
        const int kind = in < uq ? 0 : in < uq + uk ? 1 : 2; // queries, keys, values: the warp's alike
        if (ENTER && at_row[t] == -2) continue;
        if (ENTER && kind && at_row[t] < 0) continue;
        const int heads = kind ? p.Hkv : p.Hq;
        const int h0 = (kind == 0 ? in : kind == 1 ? in - uq : in - uq - uk) * kUnitRows<LANES> + group;
        const QkRows &from = kind == 0 ? q : kind == 1 ? k : v;
        const T *src = static_cast<const T *>(from.p) + (size_t)(first + t) * from.stride;
        const Place at = kind == 2 ? Place{2 * l, 2 * l + 1, false} : place_of<HALF>(l, p.rot);
        Raw16<T> raw[kUnroll] = {};
#pragma unroll
        for (int y = 0; y < kUnroll; ++y)
            if (h0 + y * GROUPS < heads) raw[y] = load16(src + (size_t)(h0 + y * GROUPS) * D, at);
        float w[16];
        if (NORM && kind < 2) load_weights(w, kind ? p.k_weight : p.q_weight, p.weight_dtype, at);
#pragma unroll
        for (int y = 0; y < kUnroll; ++y) {
            const int h = h0 + y * GROUPS;
            float x[16];
            widen16(raw[y], x);
            if (NORM && kind < 2) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
                const float r = rsqrtf(fmaf(row_sum<LANES>(sum), 1.f / D, p.eps));
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
            }
            if (at.turned) turn16<HALF>(x, turns.t[t], l, back);
            if constexpr (ENTER) {
                if (kind) {
                    const size_t row = (size_t)at_row[t] + ((size_t)h << to.c.page_shift);
                    put_rows<D>(x, at, h < heads, kind == 1 ? to.c.k : to.c.v, kind == 1 ? to.c.k_exp : to.c.v_exp,
                                to.cache_dtype, row, tops[warp]);
                    continue;
                }
            }
            const QkRows &dst = kind ? k_out : q_out;
            if (h < heads)
                store16(static_cast<T *>(const_cast<void *>(dst.p)) + (size_t)(first + t) * dst.stride + (size_t)h * D, at, x);
        }
    }
}

// The backward of a norm and its rotation: a fixed number of CTAs, which take
// every gridDim.x-th step of tokens, so that each leaves one partial sum of the
// weights' gradients; they are joined in order.  A lane adds up its 16 columns in
// registers for the queries of a step, then for the keys, and puts what it has
// into a place of its own in shared memory in between (both sums in registers
// would spill).
template <int D, bool HALF, typename T>
__global__ void __launch_bounds__(kThreads, 2)
    qk_backward_kernel(QkProblem p, QkRows q, QkRows k, QkRows dq_out, QkRows dk_out, QkRows dq, QkRows dk, float *part,
                       int step)
{
    constexpr int LANES = D / 16, GROUPS = 32 / LANES, U = sizeof(T) == 2 ? 2 : 1;
    __shared__ Turns turns;
    __shared__ __align__(16) float sums[2][4][kThreads][4]; // [kind][of 16 columns][thread]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, group = lane / LANES;
    const Place at = place_of<HALF>(l, p.rot);
    const long long tokens = (long long)p.B * p.L;
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<float4 *>(sums[i >> 2][i & 3][threadIdx.x]) = make_float4(0.f, 0.f, 0.f, 0.f);
    for (long long first = (long long)blockIdx.x * step; first < tokens; first += (long long)gridDim.x * step) {
        const int n = (int)min((long long)step, tokens - first);
        fill_turns(turns, p, first, n);
        __syncthreads();
#pragma unroll 1
        for (int kind = 0; kind < 2; ++kind) {
            const int heads = kind ? p.Hkv : p.Hq, units = units_of<LANES, U>(heads);
            const QkRows &xs = kind ? k : q, &gs = kind ? dk_out : dq_out, &ds = kind ? dk : dq;
            float w[16], acc[16] = {};
            load_weights(w, kind ? p.k_weight : p.q_weight, p.weight_dtype, at);
#pragma unroll 1
            for (int u = warp; u < n * units; u += kWarps) {
                const int t = u / units, h0 = (u - t * units) * kUnitRows<LANES, U> + group;
                const T *xp = static_cast<const T *>(xs.p) + (size_t)(first + t) * xs.stride;
                const T *gp = static_cast<const T *>(gs.p) + (size_t)(first + t) * gs.stride;
                Raw16<T> xr[U] = {}, gr[U] = {};
#pragma unroll
                for (int y = 0; y < U; ++y)
                    if (h0 + y * GROUPS < heads) {
                        xr[y] = load16(xp + (size_t)(h0 + y * GROUPS) * D, at);
                        gr[y] = load16(gp + (size_t)(h0 + y * GROUPS) * D, at);
                    }
#pragma unroll
                for (int y = 0; y < U; ++y) {
                    const int h = h0 + y * GROUPS;
                    float z[16], g[16], sum = 0.f, dot = 0.f;
                    widen16(xr[y], z);
                    widen16(gr[y], g);
                    if (at.turned) turn16<HALF>(g, turns.t[t], l, true);
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum = fmaf(z[i], z[i], sum);
                    const float r = rsqrtf(fmaf(row_sum<LANES>(sum), 1.f / D, p.eps));
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        z[i] *= r;
                        acc[i] = fmaf(g[i], z[i], acc[i]);
                        g[i] *= w[i];
                        dot = fmaf(g[i], z[i], dot);
                    }
                    dot = row_sum<LANES>(dot) * (1.f / D);
#pragma unroll
                    for (int i = 0; i < 16; ++i) z[i] = r * (g[i] - z[i] * dot);
                    if (h < heads)
                        store16(static_cast<T *>(const_cast<void *>(ds.p)) + (size_t)(first + t) * ds.stride + (size_t)h * D, at, z);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float4 *s = reinterpret_cast<float4 *>(sums[kind][i][threadIdx.x]);
                const float4 o = *s;
                *s = make_float4(o.x + acc[4 * i], o.y + acc[4 * i + 1], o.z + acc[4 * i + 2], o.w + acc[4 * i + 3]);
            }
        }
        __syncthreads(); // the table is free again
    }
    // ---- this CTA's sums: all threads that have a column
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        const int kind = i / D, col = i % D, eight = col / 8;
        // the lane that has it, and where among its 16
        int lane_of = eight / 2, in = (eight & 1) * 8 + col % 8;
        if (HALF && eight * 8 < p.rot) lane_of = eight % (p.rot / 16), in = (eight >= p.rot / 16 ? 8 : 0) + col % 8;
        float x = 0.f;
        for (int th = lane_of; th < kThreads; th += LANES) x += sums[kind][in >> 2][th][in & 3];
        part[(size_t)blockIdx.x * 2 * D + i] = x;
    }
}

// Joins n partial sums of 2 D columns each, 32 columns to a CTA.
__global__ void __launch_bounds__(kThreads)
    qk_join_kernel(const float *__restrict__ part, int n, int D, float *dq_weight, float *dk_weight)
{
    __shared__ float s[kWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = blockIdx.x * 32 + lane;
    await_previous();
    float x = 0.f;
    for (int i = warp; i < n; i += kWarps) x += part[(size_t)i * 2 * D + col];
    s[warp][lane] = x;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) x += s[w][lane];
    float *to = col < D ? dq_weight : dk_weight;
    if (to) to[col < D ? col : col - D] = x;
}

// Tokens of a CTA's step: as many as leave every SM several CTAs.
int step_for(long long tokens)
{
    int step = 1;
    while (step < kQkTokens && tokens > (long long)step * 152 * 4) step *= 2;
    return step;
}

// go(D, HALF, T) for the problem's
template <class F>
cudaError_t by_type(const QkProblem &p, int dtype, F go)
{
    auto sized = [&](auto t) {
        using T = decltype(t);
        auto laid = [&](auto d) {
            return p.interleaved ? go(d, std::false_type{}, T{}) : go(d, std::true_type{}, T{});
        };
        return p.D == 64 ? laid(std::integral_constant<int, 64>{}) : laid(std::integral_constant<int, 128>{});
    };
    return dtype == RA_BF16 ? sized(__nv_bfloat16{}) : sized(float{});
}

template <class TO>
cudaError_t forward(const QkProblem &p, int dtype, bool norm, QkRows q, QkRows k, QkRows v, QkRows q_out, QkRows k_out,
                    const TO &to, cudaStream_t s)
{
    const long long tokens = (long long)p.B * p.L;
    const int step = step_for(tokens);
    return by_type(p, dtype, [&](auto d, auto half, auto t) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        constexpr bool HALF = decltype(half)::value;
        auto kern = norm ? qk_forward_kernel<D, HALF, true, T, TO> : qk_forward_kernel<D, HALF, false, T, TO>;
        kern<<<(unsigned)((tokens + step - 1) / step), kThreads, 0, s>>>(p, q, k, v, q_out, k_out, to, step);
        return cudaGetLastError();
    });
}

} // namespace

cudaError_t launch_qk_fwd(const QkProblem &p, int dtype, bool norm, QkRows q, QkRows k, QkRows q_out, QkRows k_out,
                          cudaStream_t s)
{
    return forward(p, dtype, norm, q, k, QkRows{}, q_out, k_out, NoCache{}, s);
}

cudaError_t launch_qk_enter(const QkProblem &p, int dtype, bool norm, QkRows q, QkRows k, QkRows v, QkRows q_out,
                            const QkEnter &to, cudaStream_t s)
{
    return forward(p, dtype, norm, q, k, v, q_out, QkRows{}, to, s);
}

cudaError_t launch_qk_bwd(const QkProblem &p, int dtype, QkRows q, QkRows k, QkRows dq_out, QkRows dk_out, QkRows dq,
                          QkRows dk, float *dq_weight, float *dk_weight, float *part, cudaStream_t s)
{
    const long long tokens = (long long)p.B * p.L;
    const int step = step_for(tokens);
    const long long steps = (tokens + step - 1) / step;
    const int ctas = (int)(steps < kQkBwdCtas ? steps : kQkBwdCtas);
    const cudaError_t e = by_type(p, dtype, [&](auto d, auto half, auto t) {
        using T = decltype(t);
        qk_backward_kernel<decltype(d)::value, decltype(half)::value, T>
            <<<ctas, kThreads, 0, s>>>(p, q, k, dq_out, dk_out, dq, dk, part, step);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(qk_join_kernel, 2 * p.D / 32, kThreads, 0, s, part, ctas, p.D, dq_weight, dk_weight);
}

} // namespace ra
