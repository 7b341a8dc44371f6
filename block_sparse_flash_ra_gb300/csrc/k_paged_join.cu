// k_paged_join.cu -- joins the partial results of the paged attention.
//
// Each CTA of the attention kernels leaves, for the rows of a segment that it
// did not see whole, the unnormalised output o, the row maximum m of the
// base-2 logits and the row sum l.  With M = max m (and the sink), the row is
//   out = sum 2^(m_i - M) o_i / L,   L = sum 2^(m_i - M) l_i + 2^(sink - M),
//   lse = (M + log2 L) ln 2,
// summed in the order of the slots, so the result is the same every time.
// A sink enters here or in the attention kernel's own final store, once.
// One CTA per query row: its 4 warps take every fourth slot and meet in
// shared memory.  Bound by latency: a few slots of D floats per row.
#include <math.h>

#include "ra_paged.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;

// The partial results of a row: CTAs c0 .. c0 + n - 1, and where they lie.
struct Slots {
    long long c0, seg;
    int n, row;
    bool opens; // the segment is the first of c0's share

    __device__ __forceinline__ size_t at(const PagedPart &part, int x) const
    {
        const long long slot = part.direct ? 2 * (c0 + x) + (x == 0 && !opens ? 1 : 0) : c0 + x + seg;
        return (size_t)slot * part.slot_rows + row;
    }
};

__device__ __forceinline__ Slots find_slots(const PagedProblem &p, const PagedPart &part, int b, int i, int h,
                                            int g)
{
    const long long per_seq = (long long)part.n_rb * p.c.Hkv;
    const int n = (part.prefix ? b * p.Lq + i : i) * p.G + g;
    const int rb = n / part.row_block;
    long long total, start, seg = (long long)rb * p.c.Hkv + h;
    int tiles;
    if (part.prefix) {
        tiles = (paged_prefix_len(p) + part.tile - 1) / part.tile;
        total = per_seq * (tiles + part.seg_cost);
        start = seg * (tiles + part.seg_cost);
    } else {
        tiles = own_tiles(p, part, b);
        long long before;
        total = per_seq * own_places_sum(p, part, b, before);
        start = per_seq * before + seg * (tiles + part.seg_cost);
        seg += per_seq * b;
    }
    Slots s{0, seg, 0, n - rb * part.row_block, false};
    if (tiles == 0) return s;
    const long long share = (total + part.ctas - 1) / part.ctas;
    const long long first = start + part.seg_cost; // place of the first tile
    s.c0 = first / share;
    s.n = (int)((first + tiles - 1) / share - s.c0) + 1;
    // a share that begins before `start` begins with another segment's tile
    s.opens = start <= s.c0 * share;
    return s;
}

template <int D, typename T>
__global__ void __launch_bounds__(kWarps * 32) paged_join_kernel(PagedProblem p, PagedPart a, PagedPart b2,
                                                                 int n_parts)
{
    constexpr int V = D / 32; // values per lane
    __shared__ float o_s[kWarps][D], m_s[kWarps], l_s[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hq = blockIdx.x % p.Hq, bi = blockIdx.x / p.Hq;
    const int b = bi / p.Lq, i = bi - b * p.Lq;
    if (i >= paged_q_len(p, b)) return;
    float o[V] = {}, m = -INFINITY, l = 0.f;
    for (int k = 0; k < n_parts; ++k) {
        const PagedPart &part = k ? b2 : a;
        const Slots s = find_slots(p, part, b, i, hq / p.G, hq % p.G);
        if (part.direct && s.n == 1) return; // stored by the attention kernel
        for (int x = warp; x < s.n; x += kWarps) {
            const size_t at = s.at(part, x);
            const float mx = part.ml[at * 2], lx = part.ml[at * 2 + 1];
            float ox[V];
#pragma unroll
            for (int j = 0; j < V; ++j) ox[j] = part.o[at * D + j * 32 + lane];
            const float top = fmaxf(m, mx), base = top == -INFINITY ? 0.f : top;
            const float f = exp2f(m - base), fx = exp2f(mx - base);
            l = l * f + lx * fx;
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = o[j] * f + ox[j] * fx;
            m = top;
        }
    }
    if (warp) {
#pragma unroll
        for (int j = 0; j < V; ++j) o_s[warp][j * 32 + lane] = o[j];
        if (lane == 0) {
            m_s[warp] = m;
            l_s[warp] = l;
        }
    }
    __syncthreads();
    if (warp) return;
    float top = m;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, m_s[w]);
    const float sink = p.sinks ? p.sinks[hq] * kLog2e : -INFINITY;
    top = fmaxf(top, sink);
    const float base = top == -INFINITY ? 0.f : top;
    const float f = exp2f(m - base);
    l = l * f + exp2f(sink - base);
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] *= f;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
        const float fw = exp2f(m_s[w] - base);
        l += l_s[w] * fw;
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] += o_s[w][j * 32 + lane] * fw;
    }
    T *out = static_cast<T *>(p.out) + (size_t)blockIdx.x * D;
#pragma unroll
    for (int j = 0; j < V; ++j) out[j * 32 + lane] = (T)(l == 0.f ? 0.f : o[j] / l);
    if (lane == 0)
        p.lse[((size_t)b * p.Hq + hq) * p.Lq + i] = l == 0.f ? -INFINITY : (base + log2f(l)) * kLn2;
}

} // namespace

cudaError_t launch_paged_join(const PagedProblem &p, const PagedPart *parts, int n_parts, int dtype,
                              cudaStream_t s)
{
    const unsigned grid = (unsigned)p.B * p.Lq * p.Hq;
    const PagedPart &a = parts[0], &b = parts[n_parts - 1];
    if (dtype == RA_BF16) {
        if (p.c.D == 64) paged_join_kernel<64, __nv_bfloat16><<<grid, kWarps * 32, 0, s>>>(p, a, b, n_parts);
        else paged_join_kernel<128, __nv_bfloat16><<<grid, kWarps * 32, 0, s>>>(p, a, b, n_parts);
    } else {
        if (p.c.D == 64) paged_join_kernel<64, float><<<grid, kWarps * 32, 0, s>>>(p, a, b, n_parts);
        else paged_join_kernel<128, float><<<grid, kWarps * 32, 0, s>>>(p, a, b, n_parts);
    }
    return cudaGetLastError();
}

} // namespace ra
