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
// all heads; then each warp takes units of one or two rows per lane group, all of
// one kind (queries, keys, values).  Rows come by cp.async two units ahead, each
// lane's through a place of its own, so that loads are in flight at all times and
// cost no registers; multiply-adds are packed in pairs.
//
// Measured, bf16, D = 128: 32768 tokens of 32 + 8 heads rotated 99 us, 6.7 TB/s,
// all of a copy's rate; with norms, 32768 tokens of 16 + 16 heads, forward 83 us
// (97%), backward 131 us (92%, the join of the weights' sums 4 of them); prompts
// of 24576 tokens, 32 + 8 + 8 heads, into a 16-bit cache 102 us (89%).  Loads into
// registers as they were needed took 101, 86, 152 and 113 us.  One token of each
// of 64 sequences: 2.4 us, 4.8 into the cache; the call around it takes 7 us of
// the host's time, and two new tensors 6 more.
#include <atomic>
#include <type_traits>

#include "ra_qk.h"
#include "ra_rows.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xffffffffu;

// Cosines and sines of a step's tokens: [token][j][lane of a row] of two pairs --
// two cosines, two sines -- so that the lanes of a row read neighbouring words.
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

// 16 values as pairs, for the packed multiply-adds: eight of c0, eight of c1.
struct Sixteen {
    float2 v[8];
    __device__ __forceinline__ float at(int i) const { return i & 1 ? v[i / 2].y : v[i / 2].x; }
};

template <typename T>
__device__ __forceinline__ Sixteen widen16(const Raw16<T> &r)
{
    const Eight a = widen(r.a), b = widen(r.b);
    Sixteen x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x.v[i] = make_float2(a.x[2 * i], a.x[2 * i + 1]);
        x.v[4 + i] = make_float2(b.x[2 * i], b.x[2 * i + 1]);
    }
    return x;
}

template <typename T>
__device__ __forceinline__ void store16(T *row, const Place &at, const Sixteen &x)
{
    Eight a, b;
#pragma unroll
    for (int i = 0; i < 8; ++i) a.x[i] = x.at(i), b.x[i] = x.at(8 + i);
    store8(row + at.c0 * 8, a);
    store8(row + at.c1 * 8, b);
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// <a, b>, and the sum of it over the lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_dot(const Sixteen &a, const Sixteen &b)
{
    float2 s = fmul2(a.v[0], b.v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) s = ffma2(a.v[i], b.v[i], s);
    float x = s.x + s.y;
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

// 1 / sqrt(mean x^2 + eps) of a row
template <int D>
__device__ __forceinline__ float row_factor(const Sixteen &x, float eps)
{
    return rsqrtf(fmaf(row_dot<D / 16>(x, x), 1.f / D, eps));
}

// Turns a lane's eight pairs by the token's angles.
template <bool HALF>
__device__ __forceinline__ void turn16(Sixteen &x, const float4 (*t)[8], int l)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 cs = t[j][l]; // of pairs 8 l + 2 j and the next
        if (HALF) {
            const float2 c = make_float2(cs.x, cs.y), s = make_float2(cs.z, cs.w), a = x.v[j], b = x.v[4 + j];
            x.v[j] = fsub2(fmul2(a, c), fmul2(b, s));
            x.v[4 + j] = ffma2(a, s, fmul2(b, c));
        } else {
            const float2 a = x.v[2 * j], b = x.v[2 * j + 1];
            x.v[2 * j] = make_float2(a.x * cs.x - a.y * cs.z, a.y * cs.x + a.x * cs.z);
            x.v[2 * j + 1] = make_float2(b.x * cs.y - b.y * cs.w, b.y * cs.y + b.x * cs.w);
        }
    }
}

__device__ __forceinline__ long long position_of(const QkProblem &p, long long token)
{
    if (p.pos) return p.pos[token];
    const long long b = token / p.L;
    return token - b * p.L + (p.start ? p.start[b] : 0) + (p.prefix_len ? *p.prefix_len : 0);
}

// Fills the table for tokens [first, first + n); the backward turns the other way.
__device__ __forceinline__ void fill_turns(Turns &turns, const QkProblem &p, long long first, int n)
{
    const int pairs = p.rot / 2;
    for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
        const int t = i / pairs, pair = i - t * pairs;
        const uint64_t turn = (uint64_t)position_of(p, first + t) * p.freq[pair];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
        float *to = reinterpret_cast<float *>(&turns.t[t][(pair & 7) >> 1][pair >> 3]) + (pair & 1);
        to[0] = c * p.amplitude;
        to[2] = p.inverse ? -s * p.amplitude : s * p.amplitude;
    }
}

// A lane's 16 weights of a norm.
__device__ __forceinline__ Sixteen load_weights(const void *from, int dtype, const Place &at)
{
    if (from && dtype == RA_BF16) return widen16(load16(static_cast<const __nv_bfloat16 *>(from), at));
    if (from) return widen16(load16(static_cast<const float *>(from), at));
    Sixteen w;
#pragma unroll
    for (int i = 0; i < 8; ++i) w.v[i] = both(1.f);
    return w;
}

// u / n and its remainder, for quotients up to kQkTokens and n below 2^18 (65536
// heads): (u + 1/2) / n lies at least 1 / (2 n) > 2^-19 from a whole number, which
// is more than fp32's error of it, 2^-22 of kQkTokens.
__device__ __forceinline__ int divide(int u, int n, float inverse, int &rest)
{
    const int t = (int)(((float)u + 0.5f) * inverse);
    rest = u - t * n;
    return t;
}

// Largest magnitude of eight values, as fp32 bits.
__device__ __forceinline__ uint32_t top8(const Sixteen &x, int first)
{
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(x.at(first + i)) & 0x7fffffffu);
    return t;
}

// Stores rows of the cache, one per group of LANES lanes (`put`: there is one),
// each lane the eights c0 and c1.  tops: the warp's, a word for each eight of its rows.
template <int D>
using Tops = uint32_t[32 / (D / 16)][D / 8];
template <int D>
__device__ __forceinline__ void put_rows(const Sixteen &x, const Place &at, bool put, const void *base, const uint8_t *exps,
                                         int dtype, size_t row, Tops<D> &tops)
{
    constexpr int LANES = D / 16;
    uint8_t *bytes = static_cast<uint8_t *>(const_cast<void *>(base)), *e8 = const_cast<uint8_t *>(exps);
    if (dtype == RA_BF16) {
        if (put) store16(reinterpret_cast<__nv_bfloat16 *>(bytes) + row * D, at, x);
        return;
    }
    const int lane = threadIdx.x & 31, l = lane % LANES;
    uint32_t t0 = top8(x, 0), t1 = top8(x, 8);
    if (dtype == RA_E4M3) {
        t0 = max(t0, t1);
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) t0 = max(t0, __shfl_xor_sync(kAll, t0, o));
        t1 = t0;
    } else {
        // a block is four eights, whichever lanes have them
        uint32_t *mine = tops[lane / LANES];
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
        for (int i = 0; i < 8; ++i) y[i] = x.at(8 * h + i) * inv;
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
template <int LANES, int U>
constexpr int kUnitRows = 32 / LANES * U;
template <int LANES, int U>
__host__ __device__ __forceinline__ int units_of(int heads)
{
    return (heads + kUnitRows<LANES, U> - 1) / kUnitRows<LANES, U>;
}

__device__ __forceinline__ void copy16(uint4 *to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() // all but the last N groups
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A lane's 16 values of a row on their way through a place of its own in shared
// memory: sizeof(T) words of 16 bytes, kThreads apart.  No other thread reads
// them, so that a wait for the thread's own copies is enough.
template <typename T>
__device__ __forceinline__ void fetch16(uint4 *slot, const T *row, const Place &at)
{
    constexpr int W = sizeof(T) / 2; // words of eight values
#pragma unroll
    for (int i = 0; i < W; ++i) {
        copy16(slot + i * kThreads, reinterpret_cast<const uint4 *>(row + at.c0 * 8) + i);
        copy16(slot + (W + i) * kThreads, reinterpret_cast<const uint4 *>(row + at.c1 * 8) + i);
    }
}
template <typename T>
__device__ __forceinline__ Sixteen fetched16(const uint4 *slot, bool there)
{
    constexpr int W = sizeof(T) / 2;
    Raw16<T> r{};
    if (there) {
#pragma unroll
        for (int i = 0; i < W; ++i) r.a.w[i] = slot[i * kThreads], r.b.w[i] = slot[(W + i) * kThreads];
    }
    return widen16(r);
}

// What the forward does with its rows: they go out, or into a cache.
struct NoCache {
};

template <int D, bool HALF, bool NORM, typename T, class TO>
__global__ void __launch_bounds__(kThreads, (sizeof(T) == 2 ? 4 : 3))
    qk_forward_kernel(QkProblem p, QkRows q, QkRows k, QkRows v, QkRows q_out, QkRows k_out, TO to, int step)
{
    constexpr bool ENTER = std::is_same<TO, QkEnter>::value;
    constexpr int LANES = D / 16, GROUPS = 32 / LANES, U = sizeof(T) == 2 ? 2 : 1, kStages = 2;
    __shared__ Turns turns;
    __shared__ uint4 ring[kStages][U * sizeof(T)][kThreads];
    __shared__ __align__(16) float weights[NORM ? 2 * D : 4];
    __shared__ long long at_row[kQkTokens]; // ENTER: the token's first row in the cache, -1: in none, -2: left out
    __shared__ __align__(16) Tops<D> tops[ENTER ? kWarps : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, group = lane / LANES;
    const long long first = (long long)blockIdx.x * step;
    const int n = (int)min((long long)step, (long long)p.B * p.L - first);
    const int uq = units_of<LANES, U>(p.Hq), uk = units_of<LANES, U>(p.Hkv), units = uq + uk + (ENTER ? uk : 0);
    const float inverse = 1.f / (float)units;
    // a unit: its token, its kind (queries, keys, values: the warp's alike), the
    // lane group's first head
    struct Unit {
        int t, kind, h0, heads;
        Place at;
    };
    auto unit_of = [&](int u) {
        Unit x;
        int in;
        x.t = divide(u, units, inverse, in);
        x.kind = in < uq ? 0 : in < uq + uk ? 1 : 2;
        x.heads = x.kind ? p.Hkv : p.Hq;
        x.h0 = (x.kind == 0 ? in : x.kind == 1 ? in - uq : in - uq - uk) * kUnitRows<LANES, U> + group;
        x.at = x.kind == 2 ? Place{2 * l, 2 * l + 1, false} : place_of<HALF>(l, p.rot);
        return x;
    };
    auto fetch = [&](int u, int stage) {
        if (u < n * units) {
            const Unit x = unit_of(u);
            const QkRows &from = x.kind == 0 ? q : x.kind == 1 ? k : v;
            const T *src = static_cast<const T *>(from.p) + (size_t)(first + x.t) * from.stride + x.h0 * D;
#pragma unroll
            for (int y = 0; y < U; ++y)
                if (x.h0 + y * GROUPS < x.heads) fetch16(&ring[stage][y * sizeof(T)][threadIdx.x], src + y * GROUPS * D, x.at);
        }
        copies_end();
    };
    if constexpr (ENTER) {
        if (to.count) { // nothing to do for tokens that are all left out
            const long long b = first / p.L, i = first - b * p.L;
            const int count = to.count[b];
            if (i + n <= p.L && i >= count) {
                if (i == 0 && threadIdx.x == 0 && count < 0) report_bad_page(to.status);
                return;
            }
        }
    }
    // the first units' rows come while the angles and places are found
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(warp + i * kWarps, i);
    if (NORM && threadIdx.x < 2 * D) {
        const void *from = threadIdx.x < D ? p.q_weight : p.k_weight;
        const int i = threadIdx.x & (D - 1);
        weights[threadIdx.x] = !from                       ? 1.f
                               : p.weight_dtype == RA_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(from)[i])
                                                           : static_cast<const float *>(from)[i];
    }
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
    int stage = 0;
#pragma unroll 1
    for (int u = warp; u < n * units; u += kWarps, stage ^= 1) {
        const Unit x = unit_of(u);
        copies_wait<kStages - 1>();
        Sixteen w;
        if (NORM && x.kind < 2) w = widen16(load16(weights + x.kind * D, x.at));
#pragma unroll
        for (int y = 0; y < U; ++y) {
            const int h = x.h0 + y * GROUPS;
            Sixteen z = fetched16<T>(&ring[stage][y * sizeof(T)][threadIdx.x], h < x.heads);
            if (ENTER && (x.kind ? at_row[x.t] < 0 : at_row[x.t] == -2)) continue;
            if (NORM && x.kind < 2) {
                const float2 r = both(row_factor<D>(z, p.eps));
#pragma unroll
                for (int i = 0; i < 8; ++i) z.v[i] = fmul2(fmul2(z.v[i], r), w.v[i]);
            }
            if (x.at.turned) turn16<HALF>(z, turns.t[x.t], l);
            if constexpr (ENTER) {
                if (x.kind) {
                    const size_t row = (size_t)at_row[x.t] + ((size_t)h << to.c.page_shift);
                    put_rows<D>(z, x.at, h < x.heads, x.kind == 1 ? to.c.k : to.c.v, x.kind == 1 ? to.c.k_exp : to.c.v_exp,
                                to.cache_dtype, row, tops[warp]);
                    continue;
                }
            }
            const QkRows &dst = x.kind ? k_out : q_out;
            if (h < x.heads)
                store16(static_cast<T *>(const_cast<void *>(dst.p)) + (size_t)(first + x.t) * dst.stride + h * D, x.at, z);
        }
        fetch(u + kStages * kWarps, stage);
    }
    copies_wait<0>();
}

// The backward of a norm and its rotation: a fixed number of CTAs, which take
// every gridDim.x-th step of tokens, so that each leaves one partial sum of the
// weights' gradients; they are joined in order.  A lane adds up its 16 columns in
// registers for the queries of a step, then for the keys, and puts what it has
// into a place of its own in shared memory in between (both sums in registers
// would spill).
template <typename T>
struct BackwardSmem {
    Turns turns[2]; // of this step and, while it is found, of the next
    float sums[2][4][kThreads][4]; // [kind][of 16 columns][thread]
    uint4 ring[2][2 * sizeof(T)][kThreads];
};

template <int D, bool HALF, typename T>
__global__ void __launch_bounds__(kThreads, 2)
    qk_backward_kernel(QkProblem p, QkRows q, QkRows k, QkRows dq_out, QkRows dk_out, QkRows dq, QkRows dk, float *part,
                       int step)
{
    constexpr int LANES = D / 16, GROUPS = 32 / LANES, kStages = 2;
    extern __shared__ __align__(16) uint8_t raw_smem[];
    BackwardSmem<T> &s = *reinterpret_cast<BackwardSmem<T> *>(raw_smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, group = lane / LANES;
    const Place at = place_of<HALF>(l, p.rot);
    const long long tokens = (long long)p.B * p.L, stride = (long long)gridDim.x * step;
    const int uq = units_of<LANES, 1>(p.Hq), uk = units_of<LANES, 1>(p.Hkv);
    const float inverse_q = 1.f / (float)max(uq, 1), inverse_k = 1.f / (float)max(uk, 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<float4 *>(s.sums[i >> 2][i & 3][threadIdx.x]) = make_float4(0.f, 0.f, 0.f, 0.f);
    // a warp's units: of a step the queries' and then the keys', steps in turn
    struct At {
        long long first;
        int n, u;
    };
    auto begin = [&](long long first) { return At{first, (int)min((long long)step, tokens - first), warp}; };
    auto settle = [&](At &x) { // on to a step that has a unit for this warp
        while (x.first < tokens && x.u >= x.n * (uq + uk)) x = begin(x.first + stride);
    };
    auto unit = [&](const At &x, int &kind, int &t) { // its head of this lane group
        int in;
        kind = x.u >= x.n * uq;
        t = kind ? divide(x.u - x.n * uq, uk, inverse_k, in) : divide(x.u, uq, inverse_q, in);
        return in * kUnitRows<LANES, 1> + group;
    };
    auto fetch = [&](const At &x, int stage) {
        if (x.first < tokens) {
            int kind, t;
            const int h = unit(x, kind, t);
            if (h < (kind ? p.Hkv : p.Hq)) {
                const QkRows &xs = kind ? k : q, &gs = kind ? dk_out : dq_out;
                fetch16(&s.ring[stage][0][threadIdx.x], static_cast<const T *>(xs.p) + (size_t)(x.first + t) * xs.stride + h * D, at);
                fetch16(&s.ring[stage][sizeof(T)][threadIdx.x], static_cast<const T *>(gs.p) + (size_t)(x.first + t) * gs.stride + h * D, at);
            }
        }
        copies_end();
    };
    At now = begin((long long)blockIdx.x * step), ahead = now;
    settle(ahead);
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
        fetch(ahead, i);
        ahead.u += kWarps;
        settle(ahead);
    }
    int stage = 0, table = 0;
    for (; now.first < tokens; now = begin(now.first + stride), table ^= 1) {
        // (the table of the step before last is free: all have passed the barrier behind it)
        const Turns &turns = s.turns[table];
        fill_turns(s.turns[table], p, now.first, now.n);
        __syncthreads();
#pragma unroll 1
        for (int kind = 0; kind < 2; ++kind) {
            const int heads = kind ? p.Hkv : p.Hq;
            const Sixteen w = load_weights(kind ? p.k_weight : p.q_weight, p.weight_dtype, at);
            const QkRows &ds = kind ? dk : dq;
            Sixteen acc = {};
#pragma unroll 1
            for (const int end = now.n * (kind ? uq + uk : uq); now.u < end; now.u += kWarps, stage ^= 1) {
                int kind_too, t;
                const int h = unit(now, kind_too, t);
                copies_wait<kStages - 1>();
                Sixteen z = fetched16<T>(&s.ring[stage][0][threadIdx.x], h < heads);
                Sixteen g = fetched16<T>(&s.ring[stage][sizeof(T)][threadIdx.x], h < heads);
                fetch(ahead, stage);
                ahead.u += kWarps;
                settle(ahead);
                if (at.turned) turn16<HALF>(g, turns.t[t], l);
                const float r = row_factor<D>(z, p.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    z.v[i] = fmul2(z.v[i], both(r));
                    acc.v[i] = ffma2(g.v[i], z.v[i], acc.v[i]);
                    g.v[i] = fmul2(g.v[i], w.v[i]);
                }
                const float2 dot = both(row_dot<LANES>(g, z) * (-1.f / D));
#pragma unroll
                for (int i = 0; i < 8; ++i) z.v[i] = fmul2(both(r), ffma2(z.v[i], dot, g.v[i]));
                if (h < heads)
                    store16(static_cast<T *>(const_cast<void *>(ds.p)) + (size_t)(now.first + t) * ds.stride + h * D, at, z);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float4 *to = reinterpret_cast<float4 *>(s.sums[kind][i][threadIdx.x]);
                const float4 o = *to;
                *to = make_float4(o.x + acc.at(4 * i), o.y + acc.at(4 * i + 1), o.z + acc.at(4 * i + 2), o.w + acc.at(4 * i + 3));
            }
        }
    }
    copies_wait<0>();
    __syncthreads();
    // ---- this CTA's sums: all threads that have a column
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        const int kind = i / D, col = i % D, eight = col / 8;
        // the lane that has it, and where among its 16
        int lane_of = eight / 2, in = (eight & 1) * 8 + col % 8;
        if (HALF && eight * 8 < p.rot) lane_of = eight % (p.rot / 16), in = (eight >= p.rot / 16 ? 8 : 0) + col % 8;
        float x = 0.f;
        for (int th = lane_of; th < kThreads; th += LANES) x += s.sums[kind][in >> 2][th][in & 3];
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
#pragma unroll 8
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
                          QkRows dk, float *dq_weight, float *dk_weight, float *part, int device, cudaStream_t s)
{
    const long long tokens = (long long)p.B * p.L;
    const int step = step_for(tokens);
    const long long steps = (tokens + step - 1) / step;
    const int ctas = (int)(steps < kQkBwdCtas ? steps : kQkBwdCtas);
    const cudaError_t e = by_type(p, dtype, [&](auto d, auto half, auto t) {
        using T = decltype(t);
        auto kern = qk_backward_kernel<decltype(d)::value, decltype(half)::value, T>;
        constexpr size_t smem = sizeof(BackwardSmem<T>);
        static std::atomic<uint64_t> set{0}; // devices whose copy of the kernel has its attribute
        const uint64_t bit = 1ull << device;
        if (!(set.load(std::memory_order_acquire) & bit)) {
            const cudaError_t a = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (a != cudaSuccess) return a;
            set.fetch_or(bit, std::memory_order_release);
        }
        kern<<<ctas, kThreads, smem, s>>>(p, q, k, dq_out, dk_out, dq, dk, part, step);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(qk_join_kernel, 2 * p.D / 32, kThreads, 0, s, part, ctas, p.D, dq_weight, dk_weight);
}

} // namespace ra
