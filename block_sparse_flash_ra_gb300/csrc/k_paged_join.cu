// k_paged_join.cu -- joins the partial results of the paged attention.
//
// Each CTA of the attention kernels leaves, for the rows of a segment that it
// did not see whole, the unnormalised output o, the row maximum m of the
// base-2 logits and the row sum l.  With M = max m (and the sink), the row is
//   out = sum 2^(m_i - M) o_i / L,   L = sum 2^(m_i - M) l_i + 2^(sink - M),
//   lse = (M + log2 L) ln 2,
// summed in the order of the slots, so the result is the same every time.
// A sink enters here or in the attention kernel's own final store, once.
// A CTA of 256 threads takes 8 rows, a thread four columns of one, or, when
// there are few rows and their partial results many, one row, whose slots
// are dealt to 8 warps that meet in shared memory.  Bound by latency, or by
// reading the slots once.  Launched so that it starts while the attention
// kernels drain (their results are waited for behind the search for slots).
// What runs behind that wait is short code, run once: two slots at a time
// and the hardware's 2^x (2^-22) took 1.5 us off a call of 2048 rows against
// four slots and exp2f.
#include <math.h>

#include "ra_paged.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;

// The partial results of a row: CTAs c0 .. c0 + n - 1, and where they lie.
struct Slots {
    int c0, seg, n, row;
    bool opens; // the segment is the first of c0's share

    __device__ __forceinline__ size_t slot(const PagedPart &part, int x) const
    {
        return part.direct ? 2 * (c0 + x) + (x == 0 && !opens ? 1 : 0) : c0 + x + seg;
    }
};

// `sums`: places of all sequences and of those before sequence b0, or null to
// add them up here.
__device__ __forceinline__ Slots find_slots(const PagedProblem &p, const PagedPart &part, const unsigned *sums, int b0,
                                            int b, int i, int h, int g)
{
    const int per_seq = part.n_rb * p.c.Hkv;
    const int n = (part.prefix ? b * p.Lq + i : i) * p.G + g;
    const int rb = n / part.row_block;
    unsigned total, start;
    int tiles, seg = rb * p.c.Hkv + h;
    if (part.prefix) {
        tiles = (paged_prefix_len(p) + part.tile - 1) / part.tile;
        total = per_seq * (tiles + part.seg_cost);
        start = seg * (tiles + part.seg_cost);
    } else {
        tiles = own_tiles(p, part, b);
        unsigned before;
        if (sums) {
            const int x = b0 + (int)(threadIdx.x & 31); // at most ROWS sequences lie between
            before = sums[1] + __reduce_add_sync(0xffffffffu, x < b ? own_places(p, part, x) : 0);
            total = per_seq * sums[0];
        } else {
            total = per_seq * own_places_sum(p, part, b, before);
        }
        start = per_seq * before + seg * (tiles + part.seg_cost);
        seg += per_seq * b;
    }
    Slots s{0, seg, 0, n - rb * part.row_block, false};
    if (tiles == 0) return s;
    const unsigned share = max((total + part.ctas - 1) / part.ctas, 1u);
    const unsigned first = start + part.seg_cost; // place of the first tile
    s.c0 = min(first / share, part.ctas - 1u);
    s.n = (int)(min((first + tiles - 1) / share, part.ctas - 1u) - s.c0) + 1;
    // a share that begins before `start` begins with another segment's tile
    s.opens = start <= s.c0 * share;
    return s;
}

// Four output columns.
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// One source's contribution to a row's (o, m, l), by every `by`-th slot from
// `from` on.
template <int D>
__device__ __forceinline__ void add_slots(const PagedPart &part, const Slots &s, int from, int by, int grp, float4 &o,
                                          float &m, float &l)
{
#pragma unroll 2
    for (int x = from; x < s.n; x += by) {
        const size_t slot = s.slot(part, x);
        const float2 ml = *reinterpret_cast<const float2 *>(part.ml + (slot * part.slot_rows + s.row) * 2);
        // rows' columns lie together, or, from kernels with a thread per row,
        // groups of four columns lie together over the rows
        const size_t at = part.by_groups ? (slot * (D / 4) + grp) * part.slot_rows + s.row
                                         : (slot * part.slot_rows + s.row) * (D / 4) + grp;
        const float4 v = reinterpret_cast<const float4 *>(part.o)[at];
        const float top = fmaxf(m, ml.x), base = finite_base(top);
        const float f = ex2_approx(m - base), fx = ex2_approx(ml.x - base);
        l = l * f + ml.y * fx;
        o = make_float4(o.x * f + v.x * fx, o.y * f + v.y * fx, o.z * f + v.z * fx, o.w * f + v.w * fx);
        m = top;
    }
}

template <int D, typename T, int ROWS>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(PagedProblem p, PagedPart a, PagedPart b2, int n_parts)
{
    constexpr int G4 = D / 4, SPLIT = kThreads / (ROWS * G4); // threads per row; shares of its slots
    static_assert(SPLIT >= 1, "a CTA holds its rows");
    __shared__ Slots slots_s[ROWS][2];
    __shared__ unsigned sums_s[2];
    __shared__ int place_s[ROWS]; // (b * Lq + i) * Hq + hq, or -1
    __shared__ float4 o_s[SPLIT > 1 ? kThreads : 1];
    __shared__ float2 ml_s[SPLIT > 1 ? SPLIT * ROWS : 1];
    // rows are numbered as the prefix has them, ((b * Lq + i) * G + g), by kv
    // head, so that neighbours share a segment
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_head = p.B * p.Lq * p.G, blocks = (per_head + ROWS - 1) / ROWS;
    const int h = blockIdx.x / blocks, n0 = (blockIdx.x - h * blocks) * ROWS;
    // many sequences: their lengths are added up once for the CTA, not for each
    // row.  Whole calls with and without: 128 sequences of up to 1024 tokens 39.9
    // and 39.8 us, 192 55.0 and 55.3, 256 70.3 and 72.3, 512 of up to 128 77 and
    // 85, 4096 620 and 1310.
    const bool many = p.B > 128;
    const int b0 = n0 / (p.Lq * p.G);
    if (many) {
        if (threadIdx.x < 2) sums_s[threadIdx.x] = 0;
        __syncthreads();
        unsigned all = 0, before = 0;
#pragma unroll 4
        for (int b = threadIdx.x; b < p.B; b += kThreads) {
            const unsigned x = own_places(p, a, b);
            all += x;
            if (b < b0) before += x;
        }
        all = __reduce_add_sync(0xffffffffu, all);
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) {
            atomicAdd(sums_s, all);
            atomicAdd(sums_s + 1, before);
        }
        __syncthreads();
    }
    if (warp < ROWS) { // a warp per row looks for its slots
        const int n = n0 + warp;
        int place = -1;
        if (n < per_head) {
            const int b = n / (p.Lq * p.G), in_seq = n - b * p.Lq * p.G, i = in_seq / p.G, g = in_seq - i * p.G;
            if (i < paged_q_len(p, b)) {
                place = (b * p.Lq + i) * p.Hq + h * p.G + g;
                for (int k = 0; k < n_parts; ++k) {
                    const PagedPart &part = k ? b2 : a;
                    const Slots s = find_slots(p, part, many ? sums_s : nullptr, b0, b, i, h, g);
                    if (part.direct && s.n == 1) place = -1; // stored by the attention kernel
                    if (lane == 0) slots_s[warp][k] = s;
                }
            }
        }
        if (lane == 0) place_s[warp] = place;
    }
    __syncthreads();
    // the attention kernels' results from here on
    await_previous();
    const int r = threadIdx.x % ROWS, grp = threadIdx.x / ROWS % G4, split = threadIdx.x / (ROWS * G4);
    const int place = place_s[r];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    if (place >= 0)
#pragma unroll 1
        for (int k = 0; k < n_parts; ++k) add_slots<D>(k ? b2 : a, slots_s[r][k], split, SPLIT, grp, o, m, l);
    if (SPLIT > 1) {
        o_s[threadIdx.x] = o;
        if (grp == 0) ml_s[split * ROWS + r] = make_float2(m, l);
        __syncthreads();
        if (split) return;
        float top = m;
#pragma unroll
        for (int x = 1; x < SPLIT; ++x) top = fmaxf(top, ml_s[x * ROWS + r].x);
        const float base = finite_base(top), f = ex2_approx(m - base);
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
        l *= f;
#pragma unroll
        for (int x = 1; x < SPLIT; ++x) {
            const float2 ml = ml_s[x * ROWS + r];
            const float4 v = o_s[x * ROWS * G4 + threadIdx.x];
            const float fx = ex2_approx(ml.x - base);
            l += ml.y * fx;
            o = make_float4(o.x + v.x * fx, o.y + v.y * fx, o.z + v.z * fx, o.w + v.w * fx);
        }
        m = top;
    }
    if (place < 0) return;
    const int hq = place % p.Hq, bi = place / p.Hq;
    if (p.sinks) {
        const float sink = p.sinks[hq] * kLog2e, base = finite_base(fmaxf(m, sink)), f = ex2_approx(m - base);
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
        l = l * f + ex2_approx(sink - base);
        m = base;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    store4(static_cast<T *>(p.out) + (size_t)place * D + grp * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (grp == 0) p.lse[((size_t)(bi / p.Lq) * p.Hq + hq) * p.Lq + bi % p.Lq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D, typename T>
cudaError_t go(const PagedProblem &p, const PagedPart *parts, int n_parts, cudaStream_t s)
{
    const PagedPart &a = parts[0], &b = parts[n_parts - 1];
    const long long per_head = (long long)p.B * p.Lq * p.G, rows = per_head * p.c.Hkv;
    // 8 rows in a CTA read whole sectors and share the search for slots; below
    // one such CTA per SM, a row's own slots are what there is to spread
    // (2048 rows: 12-24 us with a row per CTA, 7-12 us with 8; 256 rows: 7 us)
    if (rows >= 8 * 152)
        return launch_dependent(paged_join_kernel<D, T, 8>, (unsigned)((per_head + 7) / 8 * p.c.Hkv), kThreads, 0, s, p, a, b,
                                n_parts);
    return launch_dependent(paged_join_kernel<D, T, 1>, (unsigned)rows, kThreads, 0, s, p, a, b, n_parts);
}

} // namespace

cudaError_t launch_paged_join(const PagedProblem &p, const PagedPart *parts, int n_parts, int dtype, cudaStream_t s)
{
    if (dtype == RA_BF16)
        return p.c.D == 64 ? go<64, __nv_bfloat16>(p, parts, n_parts, s) : go<128, __nv_bfloat16>(p, parts, n_parts, s);
    return p.c.D == 64 ? go<64, float>(p, parts, n_parts, s) : go<128, float>(p, parts, n_parts, s);
}

} // namespace ra
