// k_paged_rows.cu -- attention over a paged cache for many query rows per kv
// head at D = 128: the shared prefix of a batch, and chunks of a prompt; bf16
// queries.  The rows are the M side of the tensor-core products.
//
// With hundreds of rows on the same keys the bound is the tensor pipe (4 D
// operations per row and key) and, nearly level with it, the exponents.  An
// item is 256 rows of one kv head -- query heads, draft tokens and, for the
// prefix, sequences side by side -- as two tiles of 128 that share every K and
// V tile: while one tile's softmax runs, the pipe computes the other's
// products (PV_A(g), S_A(g+1), PV_B(g), S_B(g+1)); a thread owns a row, and P
// goes back to TMEM over the S it came from.
//
//   warps 0-7, 8-15 softmax of tiles A and B, two threads to a row, 64 keys of
//                   a tile each; they also gather the rows of Q into shared
//                   memory and store the results
//   warps 16-19     8-bit caches: widen K tiles to f16
//   warps 20-23     the same for V; 16-bit caches: clear the values behind a
//                   sequence's end
//   warps 24, 25    load K and V (a lane per page); warp 26 issues the products
// TMEM: S_A [0,128), S_B [128,256), O_A [256,384), O_B [384,512).
//
// 8-bit caches: codes times a power of two are exact in f16, so a key becomes
// code * 2^(e - E) with E the largest exponent of its tile, which then scales
// the tile's logits as one number; a value becomes
// code * 2^(e_v - EV), EV one exponent for the whole segment (raised, and O
// rescaled, when a tile's largest passes it by 2^7; f16 holds 448 * 2^7).
// What f16 loses is below 2^-32 of the largest.  The rows of Q are scaled by a
// power of two into f16's range, and P is f16 (2^-11 relative; weights below
// 2^-16 of the row's reference lose bits, below 2^-26 all of them).  References
// are whole numbers, so weights that were stored before one moved are rescaled
// by a power of two, which rounds nothing while they are normal.  Widening costs
// 1.6 instructions per pair and 96 KB of shared-memory traffic per tile of
// 2048 tensor cycles; the alternative, e4m3 terms for P as the M side of the
// few-row kernel uses, has no room in a compute-bound loop.
// 16-bit caches: the tiles go to the products as they are, P is bf16 (2^-8).
// Logits, maxima, sums and O are fp32.
//
// Measured, 512 rows on each of 8 kv heads: a prefix of 131072 e4m3 tokens
// 243 us, 61% of the bf16 rate (the softmax's exponents and conversions keep
// the pipe waiting); of 32768 tokens 89 us, 42%: some 16K cycles to the first
// product (set-up, the rows gathered, code that has not run yet), 5K to store 128 KB of
// partial results, and the join.
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "ra_paged.cuh"
#include "ra_sched.cuh"

namespace ra {
namespace {

constexpr int kKeys = 128, kHalf = 64, kD = 128;
constexpr int kThreads = 864;
constexpr int kWideWarpK = 16, kWideWarpV = 20, kLoadWarp = 24, kMmaWarp = 26;
// The softmax of 32 keys takes the row's present reference for granted:
// weights are computed at once, and only when a logit passes the reference by
// 2^13 (2^16 in bf16) -- one barrier with an or over the two warps of 32 rows
// -- is it raised, O rescaled and the 32 keys computed again from S, which their
// weights have not yet overwritten.  Two threads to a row halve the chain from
// S to P, which the ping-pong of two tiles does not hide (one thread per row
// took 2200 cycles of a tile's 4000; the products need 2460).

template <bool FP8>
struct Cfg {
    static constexpr int kMat = kKeys * kD * 2; // a 16-bit tile, 32 KB: two blocks of 128 rows x 128 bytes
    static constexpr int kRaw = kHalf * kD;     // half a tile of codes
    static constexpr int kRaws = FP8 ? 4 : 0;   // K low, K high, V low, V high of a tile, in turn
    static constexpr int kQOff = 0;
    static constexpr int kKOff = 2 * kMat;
    static constexpr int kVOff = kKOff + 2 * kMat;
    static constexpr int kRawOff = kVOff + 2 * kMat;
    // scale bytes of K tiles [2] and V tiles [2]: a tile's come before its second half
    static constexpr int kExpOff = kRawOff + kRaws * kRaw;
    static constexpr int kBarOff = kExpOff + (FP8 ? 4 * kKeys : 0);
    // k_full[2], k_empty[2], v_full[2], v_empty[2], raw_full[4], raw_empty[4],
    // q_full[2], s_full[2], p_full[2], o_full[2], v_clear[2], ev_full[4],
    // e_full[4], drain
    static constexpr int kNumBars = 8 + 8 + 10 + 4 + 4 + 1;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8 + 8;
    static constexpr int kScaleOff = kMiscOff + 16; // E of K tiles [4], EV of V tiles [4]
    static constexpr int kPairOff = kScaleOff + 48; // [tile][half][128] of the threads of a row
    static constexpr int kSmem = kPairOff + 2 * 2 * 128 * 4;
    static_assert(kSmem <= 232448 && kMiscOff % 16 == 0, "shared memory");
    static constexpr uint32_t kFmt = FP8 ? 0u : (1u << 7) | (1u << 10); // f16 or bf16 operands
    static constexpr uint32_t kIdescS = (1u << 4) | kFmt | (128u >> 3 << 17) | (128u >> 4 << 24);
    static constexpr uint32_t kIdescO = kIdescS | (1u << 16); // V is MN-major
    // Weights are 2^kPBias at the row's reference and may grow to kMost (2^15,
    // 2^16): f16 holds 2^15 and keeps all bits down to 2^-14; bf16 has fp32's range,
    // but O's sums of weights times values need some of it.
    static constexpr float kPBias = FP8 ? 2.f : 0.f, kMost = FP8 ? 32768.f : 65536.f;
};

struct Bars {
    uint64_t *k_full, *k_empty, *v_full, *v_empty, *raw_full, *raw_empty, *q_full, *s_full, *p_full, *o_full,
        *v_clear, *ev_full, *e_full, *drain;
};

template <class C>
__device__ __forceinline__ Bars carve(uint8_t *smem)
{
    Bars b;
    b.k_full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    b.k_empty = b.k_full + 2;
    b.v_full = b.k_empty + 2;
    b.v_empty = b.v_full + 2;
    b.raw_full = b.v_empty + 2;
    b.raw_empty = b.raw_full + 4;
    b.q_full = b.raw_empty + 4;
    b.s_full = b.q_full + 2;
    b.p_full = b.s_full + 2;
    b.o_full = b.p_full + 2;
    b.v_clear = b.o_full + 2;
    b.ev_full = b.v_clear + 2;
    b.e_full = b.ev_full + 4; // by raw stage: K [2], V [2]
    b.drain = b.e_full + 4;
    return b;
}

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <bool FP8>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    if (!FP8) return pack_bf16x2(lo, hi);
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 2^(b - e) of a scale byte b as a pair of halves; NaN for a row without a value
__device__ __forceinline__ __half2 half_scale(uint32_t b, int e)
{
    const int d = (int)b - e;
    return __float2half2_rn(b == 255u ? __uint_as_float(0x7fc00000u) : d < -126 ? 0.f : __uint_as_float((uint32_t)(127 + d) << 23));
}

// Rows [row0, row0 + 64) of a 16-bit tile from half a tile of codes, by 4
// warps.  A thread takes 16 codes: lanes 0-3 of a group of 8 a row's four
// chunks, lanes 4-7 those of the row 5 apart (by exclusive or), which puts the
// eight 16-byte accesses of a shared-memory phase on different banks both in
// the codes (one 128-byte row, chunks permuted by the row) and in the f16 tile
// (two per chunk).  Rows from `valid` on become 0.
__device__ __forceinline__ void widen_half(uint32_t tile, uint32_t raw, const uint8_t *exps, int row0, int valid, int e,
                                           int warp, int lane)
{
    const int x = lane & 3, in8 = (lane >> 3) ^ (lane & 4 ? 5 : 0);
#pragma unroll 1
    for (int jg = 0; jg < 2; ++jg) {
        const int j = (warp * 2 + jg) * 8 + in8; // row of the half tile
        const __half2 s = half_scale(exps[j], e);
        const bool live = row0 + j < valid;
#pragma unroll
        for (int it = 0; it < 2; ++it) { // chunks of codes x and 4 + x
            const uint4 w = lds128(raw + j * 128 + (((it * 4 + x) ^ (j & 7)) << 4));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const uint32_t h = e4m3x2_to_f16x2(y & 1 ? u[y >> 1] >> 16 : u[y >> 1] & 0xffffu);
                const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&h), s);
                o[y] = *reinterpret_cast<const uint32_t *>(&r);
            }
            if (!live) {
#pragma unroll
                for (int y = 0; y < 8; ++y) o[y] = 0u;
            }
            const uint32_t at = tile + it * (kKeys * 128) + (row0 + j) * 128;
            sts128(at + (((2 * x) ^ (j & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
            sts128(at + (((2 * x + 1) ^ (j & 7)) << 4), make_uint4(o[4], o[5], o[6], o[7]));
        }
    }
}

// The least scale that a half is is 2^-24, but codes of 448 times 2^-33 are
// still halves: the rows of a half tile that lie so far below its exponent are
// widened again, with their scale in two steps, the first of which is exact.
constexpr int kHalfLeast = 24, kFarStep = 12;
__device__ __noinline__ void widen_far(uint32_t tile, uint32_t raw, const uint8_t *exps, int row0, int valid, int e,
                                       int warp, int lane)
{
    const int x = lane & 3, in8 = (lane >> 3) ^ (lane & 4 ? 5 : 0); // as in widen_half
#pragma unroll 1
    for (int jg = 0; jg < 2; ++jg) {
        const int j = (warp * 2 + jg) * 8 + in8;
        const int d = (int)exps[j] - e;
        if (row0 + j >= valid || d >= -kHalfLeast) continue;
        const __half2 s1 = half_scale(127 - kFarStep, 127), s2 = half_scale(exps[j], e - kFarStep);
#pragma unroll 1
        for (int it = 0; it < 2; ++it) {
            const uint4 w = lds128(raw + j * 128 + (((it * 4 + x) ^ (j & 7)) << 4));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const uint32_t h = e4m3x2_to_f16x2(y & 1 ? u[y >> 1] >> 16 : u[y >> 1] & 0xffffu);
                const __half2 r = __hmul2(__hmul2(*reinterpret_cast<const __half2 *>(&h), s1), s2);
                o[y] = *reinterpret_cast<const uint32_t *>(&r);
            }
            const uint32_t at = tile + it * (kKeys * 128) + (row0 + j) * 128;
            sts128(at + (((2 * x) ^ (j & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
            sts128(at + (((2 * x + 1) ^ (j & 7)) << 4), make_uint4(o[4], o[5], o[6], o[7]));
        }
    }
}

// 32 stored weights of every thread times f, a power of two; in two steps where
// it is no half itself.  Rare, so kept out of the loop's code.
template <bool FP8>
__device__ __noinline__ void scale_stored(uint32_t at, float f)
{
    const float f1 = FP8 ? fmaxf(f, 1.f / 4096.f) : f, f0 = f < f1 ? f * 4096.f : 1.f;
    const uint32_t a = pack16<FP8>(f1, f1), b = pack16<FP8>(f0, f0);
    float w[16];
    uint32_t u[16];
    tmem_ld16(at, w);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        u[j] = __float_as_uint(w[j]);
        if (FP8) {
            const __half2 r = __hmul2(__hmul2(*reinterpret_cast<const __half2 *>(&u[j]), *reinterpret_cast<const __half2 *>(&a)),
                                      *reinterpret_cast<const __half2 *>(&b));
            u[j] = *reinterpret_cast<const uint32_t *>(&r);
        } else {
            u[j] = mul_bf16x2(u[j], a);
        }
    }
    tmem_st16(at, u);
}

template <bool FP8, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      PagedProblem p, PagedPart part)
{
    using C = Cfg<FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const Bars bars = carve<C>(smem);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kMiscOff + 4);
    const WaitCtx ctx{abort_flag, p.status, p.timeout_ns};
    // E and EV by tile mod 4: K of tile g + 4 is widened only after P V of tile
    // g + 1, EV of tile g + 4 found only after P V of tile g + 1, and both
    // softmaxes of g precede that
    volatile int *k_scale = reinterpret_cast<volatile int *>(smem + C::kScaleOff);
    volatile int *v_scale = k_scale + 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bars.k_full + s, FP8 ? 128 : 1);
            mbar_init(bars.k_empty + s, 1);
            mbar_init(bars.v_full + s, FP8 ? 128 : 1);
            mbar_init(bars.v_empty + s, 1);
            mbar_init(bars.q_full + s, 256);
            mbar_init(bars.s_full + s, FP8 ? 2 : 1);
            mbar_init(bars.p_full + s, 256);
            mbar_init(bars.o_full + s, 1);
            mbar_init(bars.v_clear + s, 128);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(bars.raw_full + s, 1);
            mbar_init(bars.raw_empty + s, 128);
            mbar_init(bars.ev_full + s, 1);
            mbar_init(bars.e_full + s, 1);
        }
        mbar_init(bars.drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    if (warp == kLoadWarp && lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    begin_in_order(part);
    report_lengths(p, part);
    PagedCursor c; // found beside the barriers' and TMEM's setting up
    const bool any = cursor_begin(p, part, blockIdx.x, c);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctx)) != 0;
    };
    auto source_len = [&](int b) { return part.prefix ? paged_prefix_len(p) : paged_kv_len(p, b); };
    // an item with at most 128 rows has no tile B
    auto two_tiles = [&](const PagedCursor &c) { return part.rows - c.rb * part.row_block > 128; };
    if (warp >= kLoadWarp) {
        if (any && warp < kMmaWarp) {
            // ------------------------------------------------------------ loads
            // a warp for K, one for V; lane x fetches box x of a half tile (codes)
            // or of a tile
            constexpr int kPart = FP8 ? kHalf : kKeys, kParts = kKeys / kPart;
            const int m = warp - kLoadWarp;
            const void *tm = m ? &tm_v : &tm_k;
            const uint8_t *exps = m ? p.c.v_exp : p.c.k_exp;
            const int box = min(p.c.page, kPart);
            uint32_t g = 0;
            bool ok = true;
            for (;;) {
                const int n = cursor_take(c), len = source_len(c.b);
                for (int t = c.t0; ok && t < c.t0 + n; ++t, ++g) {
                    const int valid = len - t * kKeys, st = g & 1;
                    // the boxes of the tile's parts: where they are in the cache
                    int z[kParts], boxes[kParts];
                    bool good[kParts];
#pragma unroll
                    for (int y = 0; y < kParts; ++y) {
                        boxes[y] = max(0, (min(valid - y * kPart, kPart) + box - 1) / box);
                        const bool mine = lane < boxes[y];
                        const int page = mine ? page_entry(p, part, c.b, t * kKeys + y * kPart + lane * box) : 0;
                        good[y] = mine && page_valid(p, page);
                        z[y] = good[y] ? page * p.c.Hkv + c.h : p.c.n_pages * p.c.Hkv; // out of range: zeros
                    }
                    const int in_page = (t * kKeys + lane * box) & (p.c.page - 1);
                    if (FP8) {
#pragma unroll
                        for (int y = 0; y < kParts; ++y) {
                            const int rs = 2 * m + y;
                            if (!(ok = wait_all(bars.raw_empty + rs, (g & 1) ^ 1))) break;
                            if (y == 0) {
                                // the tile's scale bytes (this stage's last user is widened)
                                uint8_t *e = smem + C::kExpOff + (2 * m + st) * kKeys + lane * box;
                                int bytes = 0;
#pragma unroll
                                for (int q = 0; q < kParts; ++q) {
                                    if (lane < boxes[q] && !good[q]) { // zeros, at a scale of one
                                        for (int j = 0; j < box; ++j) e[q * kPart + j] = 127;
                                        proxy_fence();
                                    }
                                    bytes += __popc(__ballot_sync(0xffffffffu, good[q])) * box;
                                }
                                if (lane == 0) mbar_expect_tx(bars.e_full + 2 * m + st, bytes);
                                __syncwarp();
#pragma unroll
                                for (int q = 0; q < kParts; ++q)
                                    if (good[q])
                                        bulk_load(e + q * kPart,
                                                  exps + ((size_t)z[q] << p.c.page_shift) + ((in_page + q * kPart) & (p.c.page - 1)), box,
                                                  bars.e_full + 2 * m + st);
                            }
                            if (lane == 0) mbar_expect_tx(bars.raw_full + rs, boxes[y] * box * kD);
                            __syncwarp();
                            if (lane < boxes[y])
                                tma_load_3d(smem + C::kRawOff + rs * C::kRaw + lane * box * 128, tm, bars.raw_full + rs, 0,
                                            (in_page + y * kPart) & (p.c.page - 1), z[y]);
                        }
                    } else {
                        if (!(ok = wait_all((m ? bars.v_empty : bars.k_empty) + st, ((g >> 1) & 1) ^ 1))) break;
                        uint64_t *full = (m ? bars.v_full : bars.k_full) + st;
                        if (lane == 0) mbar_expect_tx(full, boxes[0] * box * kD * 2);
                        __syncwarp();
                        uint8_t *dst = smem + (m ? C::kVOff : C::kKOff) + st * C::kMat + lane * box * 128;
                        if (lane < boxes[0])
                            for (int hf = 0; hf < 2; ++hf)
                                tma_load_3d(dst + hf * (kKeys * 128), tm, full, hf * 64, in_page, z[0]);
                    }
                }
                if (!ok || !cursor_next(p, part, c, n)) break;
            }
            if (!ok) {
                // copies on their way land before the CTA ends (a phase that
                // passed already, or was not begun, only runs the clock)
                for (int s = 0; s < 2; ++s)
                    for (uint32_t x = 0; x < 2 && x <= g; ++x) {
                        const uint32_t two = ((g - x) >> 1) & 1;
                        if (FP8) {
                            wait_drain(bars.raw_full + 2 * m + s, (g - x) & 1, kDrainNs);
                            wait_drain(bars.e_full + 2 * m + s, two, kDrainNs);
                        } else {
                            wait_drain((m ? bars.v_full : bars.k_full) + s, two, kDrainNs);
                        }
                    }
            }
        } else if (any && warp == kMmaWarp) {
            // ------------------------------------------------------------ products
            const uint64_t qd0 = sdesc_sw128(smem_u32(smem + C::kQOff), 16, 1024);
            const uint64_t kd0 = sdesc_sw128(smem_u32(smem + C::kKOff), 16, 1024);
            const uint64_t vd0 = sdesc_sw128(smem_u32(smem + C::kVOff), kKeys * 128, 1024);
            constexpr uint32_t kStep = C::kMat >> 4;
            uint32_t g = 0, segs = 0, segs_b = 0, parts_b = 0;
            bool ok = true;
            auto issue_s = [&](int x, uint32_t j) {
                const uint64_t qd = qd0 + (uint32_t)(x * kStep), kd = kd0 + (j & 1) * kStep;
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * (kKeys * 128) + (kk & 3) * 32) >> 4;
                    mma_ss_w(tmem + x * 128, qd + o, kd + o, C::kIdescS, kk > 0 ? 1u : 0u);
                }
                // the softmax reads the tile's E as well as S: this arrival passes on
                // what the wait for the wide tile has seen
                if (FP8 && lane == 0) mbar_arrive(bars.s_full + x);
                tc_commit_w(bars.s_full + x);
            };
            auto issue_pv = [&](int x, uint32_t j, uint32_t ph, bool first) -> bool {
                const uint64_t vd = vd0 + (j & 1) * kStep;
                if (!wait_all(bars.p_full + x, ph)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ts_w(tmem + 256 + x * 128, tmem + x * 128 + (kk >> 2) * 64 + (kk & 3) * 8, vd + (uint32_t)((kk * 2048) >> 4),
                             C::kIdescO, (kk > 0 || !first) ? 1u : 0u);
                return true;
            };
            for (;;) {
                const int n = cursor_take(c);
                const bool both = two_tiles(c);
                // first S products of the segment
                if (!(ok = wait_all(bars.q_full + 0, segs++ & 1))) break;
                if (both && !(ok = wait_all(bars.q_full + 1, segs_b++ & 1))) break;
                if (!(ok = wait_all(bars.k_full + (g & 1), (g >> 1) & 1))) break;
                tc_fence_after();
                issue_s(0, g);
                if (both) issue_s(1, g);
                tc_commit_w(bars.k_empty + (g & 1));
                for (int t = 0; t < n; ++t, ++g) {
                    const bool more = t + 1 < n;
                    if (!(ok = wait_all((FP8 ? bars.v_full : bars.v_clear) + (g & 1), (g >> 1) & 1))) break;
                    if (!(ok = issue_pv(0, g, g & 1, t == 0))) break;
                    if (!more) tc_commit_w(bars.o_full + 0);
                    if (more) {
                        if (!(ok = wait_all(bars.k_full + ((g + 1) & 1), ((g + 1) >> 1) & 1))) break;
                        tc_fence_after();
                        issue_s(0, g + 1);
                    }
                    if (both) {
                        if (!(ok = issue_pv(1, g, parts_b++ & 1, t == 0))) break;
                        if (!more) tc_commit_w(bars.o_full + 1);
                    }
                    tc_commit_w(bars.v_empty + (g & 1));
                    if (more) {
                        if (both) issue_s(1, g + 1);
                        tc_commit_w(bars.k_empty + ((g + 1) & 1));
                    }
                }
                if (!ok || !cursor_next(p, part, c, n)) break;
            }
            tc_commit_w(bars.drain);
            wait_drain(bars.drain, 0, kDrainNs);
        }
    } else if (warp >= kWideWarpK) {
        // ---------------------------------------------------------------- tiles
        const int w = warp & 3, st_raw = warp >= kWideWarpV ? 2 : 0;
        const uint32_t raw = smem_u32(smem + C::kRawOff + st_raw * C::kRaw);
        uint64_t *raw_full = bars.raw_full + st_raw, *raw_empty = bars.raw_empty + st_raw;
        uint32_t g = 0;
        bool ok = true;
        while (any && ok) {
            const int n = cursor_take(c), len = source_len(c.b);
            int ev = -1; // EV of the segment
            for (int t = c.t0; ok && t < c.t0 + n; ++t, ++g) {
                const int valid = min(len - t * kKeys, kKeys), st = g & 1;
                if (!FP8) {
                    if (st_raw == 0) continue;
                    // values behind the length: whatever is there, weight 0 must give 0
                    if (!(ok = wait_all(bars.v_full + st, (g >> 1) & 1))) break;
                    const int j = threadIdx.x - kWideWarpV * 32;
                    if (j >= valid)
                        for (int x = 0; x < 16; ++x)
                            sts128(smem_u32(smem + C::kVOff + st * C::kMat) + (x >> 3) * (kKeys * 128) + j * 128 + (x & 7) * 16,
                                   make_uint4(0, 0, 0, 0));
                    if (valid < kKeys) proxy_fence();
                    mbar_arrive(bars.v_clear + st);
                } else {
                    const uint32_t tile = smem_u32(smem + (st_raw ? C::kVOff : C::kKOff) + st * C::kMat);
                    const uint8_t *ex = smem + C::kExpOff + (st_raw + st) * kKeys;
                    if (!(ok = wait_all(bars.e_full + st_raw + st, (g >> 1) & 1))) break;
                    // the tile's largest exponent (1 at least: its float is normal);
                    // rows without a value do not count
                    int top = 1, low = 255;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int j = lane + 32 * y, b = ex[j];
                        if (j < valid && b != 255) top = max(top, b), low = min(low, b);
                    }
                    int e = (int)__reduce_max_sync(0xffffffffu, (unsigned)top);
                    if (st_raw) {
                        // values keep the segment's: 448 * 2^7 is the most that f16 holds
                        if (ev >= 0 && e <= ev + 7) e = ev;
                        ev = e;
                    }
                    if (w == 0 && lane == 0) {
                        (st_raw ? v_scale : k_scale)[g & 3] = e;
                        // the softmax needs EV, but not the values
                        if (st_raw) mbar_arrive(bars.ev_full + (g & 3));
                    }
                    const bool far = __any_sync(0xffffffffu, low < e - kHalfLeast);
                    if (!(ok = wait_all((st_raw ? bars.v_empty : bars.k_empty) + st, ((g >> 1) & 1) ^ 1))) break;
#pragma unroll 1
                    for (int y = 0; y < 2 && ok; ++y) {
                        if (!(ok = wait_all(raw_full + y, g & 1))) break;
                        widen_half(tile, raw + y * C::kRaw, ex + y * kHalf, y * kHalf, valid, e, w, lane);
                        if (far) widen_far(tile, raw + y * C::kRaw, ex + y * kHalf, y * kHalf, valid, e, w, lane);
                        mbar_arrive(raw_empty + y);
                    }
                    if (!ok) break;
                    proxy_fence();
                    mbar_arrive((st_raw ? bars.v_full : bars.k_full) + st);
                }
            }
            if (!ok || !cursor_next(p, part, c, n)) break;
        }
    } else {
        // ---------------------------------------------------------------- softmax
        // From the first wait that gave up on, a thread makes no wait any more
        // and runs its loops out on whatever is there: the barrier of two warps
        // is still met by all of their threads, converged.
        const int x = warp >> 3, y = (warp >> 2) & 1; // tile A or B; keys 64 y .. 64 y + 63
        const int row_in = (warp & 3) * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_half = lane_base + x * 128 + y * 64, o_half = lane_base + 256 + x * 128 + y * 64;
        float *pair = reinterpret_cast<float *>(smem + C::kPairOff) + x * 256 + row_in; // + 128 for the other half
        const float cap2 = p.soft_cap * kLog2e, to_cap = p.soft_cap > 0.f ? kLn2 / p.soft_cap : 0.f;
        uint32_t g = 0, gx = 0, segs = 0;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = mbar_wait(bar, parity, ctx);
            __syncwarp();
        };
        // the two warps of 32 rows meet
        const int pair_bar = 1 + x * 4 + (warp & 3);
        auto pair_sync = [&]() { asm volatile("barrier.sync %0, 64;" ::"r"(pair_bar) : "memory"); };
        auto pair_or = [&](bool v) {
            uint32_t r;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                         "barrier.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(r)
                         : "r"((uint32_t)v), "r"(pair_bar)
                         : "memory");
            return r != 0;
        };
        while (any) {
            const int n = cursor_take(c), len = source_len(c.b);
            const bool mine = x == 0 || two_tiles(c); // uniform over the tile's threads
            int limit = len; // keys that the row sees
            // ---- Q: 16 lanes take a row, 8 values each; a warp loads 16 rows,
            // the other half's warp the other 16
            float a_row = p.scale * kLog2e;
            if (mine) {
                const PagedRow row = paged_row(p, part, c, x * 128 + row_in);
                const int place = row.counts ? (row.b * p.Lq + row.i) * p.Hq + c.h * p.G + row.g : -1;
                if (row.counts) limit = min(row.limit, len);
                const int ch = lane & 15;
                uint4 u[8];
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                    const int src = __shfl_sync(0xffffffffu, place, y * 16 + 2 * it + (lane >> 4));
                    u[it] = make_uint4(0, 0, 0, 0);
                    if (src >= 0)
                        u[it] = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + (size_t)src * kD)[ch];
                }
#pragma unroll 1
                for (int it = 0; it < 8; it += 2) { // one piece of code for all
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int r_in = (warp & 3) * 32 + y * 16 + 2 * (it + z) + (lane >> 4);
                        uint32_t v[4] = {u[z].x, u[z].y, u[z].z, u[z].w};
                        if (FP8) {
                            // largest magnitude, as bf16 bits, two at a time
                            const uint32_t m = 0x7fff7fffu;
                            uint32_t top = __vmaxu2(__vmaxu2(v[0] & m, v[1] & m), __vmaxu2(v[2] & m, v[3] & m));
#pragma unroll
                            for (int o = 1; o < 16; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
                            top = max(top & 0xffffu, top >> 16);
                            const int e = top == 0 ? 0 : min(max((int)(top >> 7) - 127, -120), 120);
                            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                v[k] = pack16<true>(__uint_as_float(v[k] << 16) * inv, __uint_as_float(v[k] & 0xffff0000u) * inv);
                            if (ch == 0) pair[r_in - row_in] = __uint_as_float((uint32_t)(127 + e) << 23);
                        }
                        sts128(smem_u32(smem + C::kQOff + x * C::kMat) + (ch >> 3) * (kKeys * 128) + r_in * 128 +
                                   (((ch & 7) ^ (r_in & 7)) << 4),
                               make_uint4(v[0], v[1], v[2], v[3]));
                    }
#pragma unroll
                    for (int k = 0; k < 6; ++k) u[k] = u[k + 2];
                }
                proxy_fence();
            }
            // (tile B's threads run ahead over segments that have none: no arrival,
            // or the barrier could pass two phases before anyone waits)
            if (mine) mbar_arrive(bars.q_full + x);
            if (FP8 && mine) {
                pair_sync();
                a_row *= pair[0];
            }
            const int all = __reduce_min_sync(0xffffffffu, limit);

            float m = -INFINITY, l = 0.f; // l: of this thread's keys
            int ev = 0;
            // this thread's half of O's columns times f (every product into O
            // has completed)
            auto scale_o = [&](float f) {
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    float o[16];
                    tmem_ld16(o_half + k * 16, o);
                    tmem_ld_wait();
                    uint32_t u[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(o[j] * f);
                    tmem_st16(o_half + k * 16, u);
                }
                tmem_st_wait();
            };
            for (int t = c.t0; mine && t < c.t0 + n; ++t, ++gx) {
                const uint32_t gt = g + (t - c.t0); // the tile's number in this CTA
                const bool masked = all < (t + 1) * kKeys;
                float a = a_row, fv = 1.f; // the tile's logit scale; the change of EV
                if (FP8) {
                    // tile B's threads come here from segments that have none without
                    // having waited in them: ev_full could be several phases behind,
                    // and its parity say nothing, before S is there
                    if (t == c.t0) wait(bars.s_full + x, gx & 1);
                    wait(bars.ev_full + (gt & 3), (gt >> 2) & 1);
                    const int e = v_scale[gt & 3];
                    if (t > c.t0 && e != ev) fv = ex2_approx((float)(ev - e));
                    ev = e;
                }
                wait(bars.s_full + x, gx & 1);
                tc_fence_after();
                if (FP8) {
                    a *= __uint_as_float((uint32_t)k_scale[gt & 3] << 23);
                    // S of this tile completed after P V of the one before
                    if (fv != 1.f) scale_o(fv);
                }
                uint32_t pk[16];
                float sum = 0.f;
                // Capped and masked logits of 16 of the thread's keys, from its key j0
                // on, in units of b.  Masked tiles are rare and have code of their own,
                // so that the common path is short and in one piece.
                const float b = CAP ? 1.f : a;
                auto logits = [&](auto masked_tag, float *v, int j0) {
                    if (CAP) {
                        // the odd series where it holds (3.4e-7 relative), two lanes
                        // per instruction; else 1 - 2 / (1 + e^2x)
                        const float a1 = a * to_cap;
                        float xa = 0.f;
#pragma unroll
                        for (int j = 0; j < 16; j += 2) xa = max3(xa, fabsf(v[j]), fabsf(v[j + 1]));
                        if (__all_sync(0xffffffffu, xa * a1 < kTanhSmall)) {
                            const float2 k1 = make_float2(a1, a1), d7 = make_float2(cap2 * kTanhC7, cap2 * kTanhC7);
                            const float2 d5 = make_float2(cap2 * kTanhC5, cap2 * kTanhC5);
                            const float2 d3 = make_float2(cap2 * kTanhC3, cap2 * kTanhC3), d1 = make_float2(cap2, cap2);
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                const float2 xx = fmul2(make_float2(v[j], v[j + 1]), k1), x2 = fmul2(xx, xx);
                                const float2 r = fmul2(xx, ffma2(x2, ffma2(x2, ffma2(x2, d7, d5), d3), d1));
                                v[j] = r.x;
                                v[j + 1] = r.y;
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = cap2 * tanh_near(v[j] * a1);
                        }
                    }
                    if (decltype(masked_tag)::value) {
                        const int seen = limit - t * kKeys - y * 64 - j0; // of the 16
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (j >= seen) v[j] = -INFINITY;
                    }
                };
                // their weights, with the exponent's offset nm
                auto weights = [&](const float *v, float nm, int k) {
                    const float2 a2 = make_float2(b, b), n2 = make_float2(nm, nm);
                    float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float2 e2 = ffma2(make_float2(v[j], v[j + 1]), a2, n2);
                        const float2 e = make_float2(ex2_approx(e2.x), ex2_approx(e2.y));
                        ls[(j >> 1) & 1] = fadd2(ls[(j >> 1) & 1], e);
                        pk[k * 8 + (j >> 1)] = pack16<FP8>(e.x, e.y);
                    }
                    const float2 l2 = fadd2(ls[0], ls[1]);
                    sum += l2.x + l2.y;
                };
                auto keys32 = [&](auto masked_tag, int q) { // the thread's keys 32 q .. 32 q + 31
                    const float nm = C::kPBias - finite_base(m);
                    sum = 0.f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float s[16];
                        tmem_ld16(s_half + q * 32 + k * 16, s);
                        tmem_ld_wait();
                        logits(masked_tag, s, q * 32 + k * 16);
                        weights(s, nm, k);
                    }
                };
                auto half = [&](auto masked_tag) {
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
#pragma unroll 1
                        for (int pass = 0;; ++pass) {
                            keys32(masked_tag, q);
                            // No weight is above kMost when their sum is not.  A first
                            // logit sets the reference, one far above it raises it.
                            if (pass || !pair_or(m == -INFINITY || !(sum <= C::kMost))) break;
                            float top = -INFINITY;
#pragma unroll 1
                            for (int k = 0; k < 2; ++k) {
                                float s[16];
                                tmem_ld16(s_half + q * 32 + k * 16, s);
                                tmem_ld_wait();
                                logits(masked_tag, s, q * 32 + k * 16);
#pragma unroll
                                for (int j = 0; j < 16; j += 2) top = max3(top, s[j], s[j + 1]);
                            }
                            pair[y * 128] = top * b;
                            pair_sync();
                            // whole numbers: f, which the 16-bit weights of the first keys are
                            // multiplied by too, is a power of two then
                            const float m_new = floorf(max3(m, top * b, pair[(y ^ 1) * 128]));
                            const float f = m == m_new ? 1.f : ex2_approx(m - m_new); // 0 for a first one
                            m = m_new;
                            l *= f;
                            if (t > c.t0) scale_o(f);
                            if (q) {
                                // the thread's first 32 keys are stored, but not handed over
                                scale_stored<FP8>(s_half, f);
                            }
                        }
                        l += sum;
                        // over columns of S that this thread is done with
                        tmem_st16(s_half + q * 16, pk);
                    }
                };
                if (masked) half(std::true_type{});
                else half(std::false_type{});
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bars.p_full + x);
            }
            g += n;
            // ---- the segment's end: this row's result, half of its columns
            if (mine) {
                wait(bars.o_full + x, segs & 1);
                ++segs;
                pair[y * 128] = l; // both threads of the row are done with its tiles
                pair_sync();
                l = pair[0] + pair[128];
                tc_fence_after();
                const PagedRow row = paged_row(p, part, c, x * 128 + row_in);
                const int hq = c.h * p.G + row.g;
                const size_t place = ((size_t)row.b * p.Lq + row.i) * p.Hq + hq;
                float mr = m - C::kPBias; // l and O are relative to 2^mr
                const bool final = stores_whole(part, c, n);
                const size_t slot = slot_row(part, c);
                const int in_slot = x * 128 + row_in;
                float f = FP8 ? __uint_as_float((uint32_t)ev << 23) : 1.f;
                if (final) {
                    if (p.sinks && row.counts) {
                        const float sink = p.sinks[hq] * kLog2e, with = finite_base(fmaxf(mr, sink)), old = ex2_approx(mr - with);
                        f *= old;
                        l = l * old + ex2_approx(sink - with);
                        mr = with;
                    }
                    f = l == 0.f ? 0.f : f / l;
                }
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    float o[16];
                    tmem_ld16(o_half + k * 16, o);
                    tmem_ld_wait();
                    const int col = y * 64 + k * 16;
                    if (row.counts && final) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + place * kD + col);
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            dst[j] = make_uint4(pack_bf16x2(o[8 * j] * f, o[8 * j + 1] * f), pack_bf16x2(o[8 * j + 2] * f, o[8 * j + 3] * f),
                                                pack_bf16x2(o[8 * j + 4] * f, o[8 * j + 5] * f), pack_bf16x2(o[8 * j + 6] * f, o[8 * j + 7] * f));
                    } else if (row.counts) {
                        // groups of four columns over the rows: a warp's rows lie together
                        float4 *dst = reinterpret_cast<float4 *>(part.o) + slot * (kD / 4) + (size_t)(col / 4) * part.slot_rows + in_slot;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            dst[j * part.slot_rows] = make_float4(o[4 * j] * f, o[4 * j + 1] * f, o[4 * j + 2] * f, o[4 * j + 3] * f);
                    }
                    __syncwarp(); // the next read of TMEM is the whole warp's
                }
                tc_fence_before();
                if (row.counts && y == 0) {
                    if (final)
                        p.lse[((size_t)row.b * p.Hq + hq) * p.Lq + row.i] = l == 0.f ? -INFINITY : (mr + log2f(l)) * kLn2;
                    else
                        *reinterpret_cast<float2 *>(part.ml + (slot + in_slot) * 2) = make_float2(mr, l);
                }
                pair_sync(); // pair is free again
            }
            if (!cursor_next(p, part, c, n)) break;
        }
    }
    await_previous();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <bool FP8, bool CAP>
cudaError_t go(const PagedProblem &p, const PagedPart &part, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s)
{
    auto kern = paged_rows_kernel<FP8, CAP>;
    static std::atomic<uint64_t> set{0}; // devices whose copy of the kernel has its attribute
    const uint64_t bit = 1ull << p.device;
    if (!(set.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<FP8>::kSmem);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_release);
    }
    return launch_dependent(kern, (unsigned)part.ctas, kThreads, Cfg<FP8>::kSmem, s, k, v, p, part);
}

} // namespace

cudaError_t launch_paged_rows(const PagedProblem &p, const PagedPart &part, int cache_dtype, const void *tm_k,
                              const void *tm_v, cudaStream_t s)
{
    const CUtensorMap &k = *static_cast<const CUtensorMap *>(tm_k), &v = *static_cast<const CUtensorMap *>(tm_v);
    if (p.soft_cap > 0.f)
        return cache_dtype == RA_E4M3 ? go<true, true>(p, part, k, v, s) : go<false, true>(p, part, k, v, s);
    return cache_dtype == RA_E4M3 ? go<true, false>(p, part, k, v, s) : go<false, false>(p, part, k, v, s);
}

} // namespace ra
