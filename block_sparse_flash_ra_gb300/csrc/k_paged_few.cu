// k_paged_few.cu -- attention over a paged cache for at most 16 query rows
// per kv head and item: decoding steps and short drafts, bf16 queries.
//
// Bound by memory: a cached byte is used by a handful of rows.  So the kernel
// is built around keeping loads in flight: each of a CTA's 4 warps takes its
// own quarter of every tile (32 keys of 8 bit, 16 of 16 bit at D = 128) and
// owns a ring of 3 stages that it fills itself with TMA copies, one stage
// ahead of the page numbers it needs next; no warp waits for another inside a
// segment, and the ring runs on across segments.  8 warps per SM keep up to
// 196 KB in flight; 6.8 TB/s over 152 SMs need some 45 KB.
//
// A warp's product is S (16 rows x 8 keys) += Q (16 x 16) K^T with
// mma.sync.m16n8k16: tcgen05 would pad the rows to 64 or 128 and would need
// the 8-bit rows widened through shared memory, while here the codes are
// widened in registers on their way into the fragments.  The contraction
// index may be permuted freely, so a thread takes 16 contiguous bytes of a
// key (or of a value: column n of O block nb is d = n * (D / 8) + nb), and
// keys within a group of 8 are permuted by kPerm so that all eight lanes of a
// shared-memory phase hit different banks of the 128-byte swizzle.
//
// 8-bit caches: codes are exact in f16; the query row is scaled by a power of
// two into f16's range (bf16 has fewer bits, so this too is exact down to
// 2^-24 of the row's maximum), the key's scale multiplies the logit, the
// value's scale multiplies the probability.  Weights p 2^(e_v - E) 2^11 are
// f16, E the largest e_v so far in the warp: 2^-11 relative, below 2^-25 of
// the largest absolute.  16-bit caches: bf16 products, with p as a sum of two
// bf16 (2^-16 relative), so that rounding p does not show in the output.
// Logits, maxima and sums are fp32; O is rescaled only when a row's maximum
// has grown by more than 2^4 (or E has grown).
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>

#include <atomic>

#include "ra_paged.cuh"
#include "ra_sched.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr float kLazy = 4.f;   // growth of a row maximum (base 2) that is let pass
constexpr float kPBias = 11.f; // 8-bit caches: weights are kept times 2^11 (2^15 with kLazy)

constexpr int D = 64;
constexpr int kKeys = 32; // keys of one stage (per warp)
constexpr int kTile = kPagedFewTile;
static_assert(kTile == kWarps * kKeys, "a warp takes a quarter of a tile");

template <bool FP8>
struct Cfg {
    static constexpr int kRowBytes = D * (FP8 ? 1 : 2); // one TMA box is this wide
    static constexpr int kMatBytes = kKeys * kRowBytes;
    static constexpr int kStageBytes = 2 * kMatBytes;
    static constexpr int kStages = kStageBytes <= 4096 ? 4 : 3;
    // per warp: the stages, then the scale bytes of each (K, V)
    static constexpr int kExpBytes = FP8 ? 2 * kKeys : 0;
    static constexpr int kExpOff = kWarps * kStages * kStageBytes;
    static constexpr int kMergeOff = kExpOff + kWarps * kStages * kExpBytes;
    static constexpr int kMergeBytes = (kWarps - 1) * 8 * D * 4;
    static constexpr int kStatOff = kMergeOff + kMergeBytes; // [4 warps][16 rows][m, l]
    static constexpr int kBarOff = kStatOff + kWarps * 16 * 8;
    static constexpr int kMiscOff = kBarOff + kWarps * kStages * 8;
    static constexpr int kSmem = kMiscOff + 16 + 1024; // slack for 1024-byte alignment
    static_assert(kSmem <= 113 * 1024, "two CTAs per SM");
};

// Key of fragment column n inside its group of 8 (see above).
__device__ __forceinline__ int key_perm(int n) { return (0x37156240 >> (4 * n)) & 7; }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, uint64_t *bar, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// c += A B.  With ROWS == 8 the lower half of A is zero and the lower half of
// the product is dropped, so that no registers are kept for it.
template <bool FP8, int ROWS>
__device__ __forceinline__ void mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    if (ROWS == 16) {
        if (FP8)
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                         "{%0,%1,%2,%3};"
                         : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
        else
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                         "{%0,%1,%2,%3};"
                         : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    } else {
        float x, y;
        if (FP8)
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%8,%5,%8}, {%6,%7}, "
                         "{%0,%1,%9,%9};"
                         : "+f"(c[0]), "+f"(c[1]), "=f"(x), "=f"(y)
                         : "r"(a[0]), "r"(a[2]), "r"(b0), "r"(b1), "r"(0), "f"(0.f));
        else
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%8,%5,%8}, {%6,%7}, "
                         "{%0,%1,%9,%9};"
                         : "+f"(c[0]), "+f"(c[1]), "=f"(x), "=f"(y)
                         : "r"(a[0]), "r"(a[2]), "r"(b0), "r"(b1), "r"(0), "f"(0.f));
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Shared-memory address of 16-byte chunk c of row j of a staged matrix.
template <bool FP8>
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int j, int c)
{
    if (FP8) return base + j * 64 + ((c ^ ((j >> 1) & 3)) << 4);
    return base + j * 128 + ((c ^ (j & 7)) << 4);
}

// What a warp loads next: its keys of one tile.
struct Ahead {
    PagedCursor c;
    int n;     // tiles of the segment that the share still has (from c.t0)
    int len;   // keys of the segment's source
    int valid; // keys of this stage (0: nothing ahead)
    int page[2]; // as the table has them
    bool live;
};

template <bool FP8, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, 2)
    paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     PagedProblem p, PagedPart part)
{
    using C = Cfg<FP8>;
    constexpr int NB = kKeys / 8;   // key groups of a stage
    constexpr int KS = D / 16;         // contraction steps of Q K^T
    constexpr int OB = D / 8;          // O blocks
    constexpr int RH = ROWS / 8;       // row halves that a thread holds
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOff) + warp * C::kStages;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kMiscOff);
    const WaitCtx ctx{abort_flag, p.status, p.timeout_ns};
    const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
    const uint32_t exps = smem_u32(smem) + C::kExpOff + warp * C::kStages * C::kExpBytes;
    float4 *merge = reinterpret_cast<float4 *>(smem + C::kMergeOff);
    float2 *stat = reinterpret_cast<float2 *>(smem + C::kStatOff);

    if (lane == 0) {
        for (int s = 0; s < C::kStages; ++s) mbar_init(bars + s, 1);
        if (warp == 0) *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    begin_in_order(part);
    report_lengths(p, part);
    __syncthreads();
    PagedCursor c;
    if (!cursor_begin(p, part, blockIdx.x, c)) {
        await_previous();
        return;
    }

    // ---- the loads ahead.  A box is as many keys as a page and a stage share.
    const int box = min(p.c.page, kKeys);
    Ahead a;
    a.c = c;
    auto source_len = [&](int b) { return part.prefix ? paged_prefix_len(p) : paged_kv_len(p, b); };
    auto onward = [&]() {
        if (--a.n > 0) {
            ++a.c.t0;
            --a.c.left;
        } else if ((a.live = cursor_next(p, part, a.c, 1))) {
            a.n = cursor_take(a.c);
            a.len = source_len(a.c.b);
        }
    };
    // finds the warp's keys of the tile at a.c (or of a later one) and starts
    // the read of their page numbers
    auto look = [&]() {
        while (a.live) {
            const int first = a.c.t0 * kTile + warp * kKeys;
            a.valid = min(a.len - first, kKeys);
            if (a.valid > 0) {
                a.page[0] = page_entry(p, part, a.c.b, first);
                if (box < kKeys && a.valid > box) a.page[1] = page_entry(p, part, a.c.b, first + box);
                return;
            }
            onward();
        }
    };
    uint32_t issued = 0;
    bool ok = true;
    // fills the next stage; a page out of range has z behind the tensor's
    // end, which the copy fills with zeros
    auto issue = [&]() {
        if (!a.live || !ok) return;
        const int s = issued % C::kStages;
        if (lane == 0) {
            const int boxes = (a.valid + box - 1) / box;
            const int first = a.c.t0 * kTile + warp * kKeys;
            const int off = first & (p.c.page - 1);
            uint8_t *eb = smem + C::kExpOff + (warp * C::kStages + s) * C::kExpBytes;
            int bytes = boxes * box * C::kRowBytes * 2;
            bool good[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                good[x] = x < boxes && page_valid(p, a.page[x]);
                if (FP8 && good[x]) bytes += 2 * box;
                if (FP8 && x < boxes && !good[x]) {
                    for (int j = 0; j < box; ++j) eb[x * box + j] = eb[kKeys + x * box + j] = 127;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
            }
            mbar_expect_tx(bars + s, bytes);
            const uint32_t dst = ring + s * C::kStageBytes;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (x >= boxes) break;
                const int z = good[x] ? a.page[x] * p.c.Hkv + a.c.h : p.c.n_pages * p.c.Hkv;
                const uint32_t at = dst + x * box * C::kRowBytes;
                tma_load_3d(at, &tm_k, bars + s, 0, off, z);
                tma_load_3d(at + C::kMatBytes, &tm_v, bars + s, 0, off, z);
                if (FP8 && good[x]) {
                    const size_t row = ((size_t)z << p.c.page_shift) + off;
                    bulk_load(eb + x * box, p.c.k_exp + row, box, bars + s);
                    bulk_load(eb + kKeys + x * box, p.c.v_exp + row, box, bars + s);
                }
            }
        }
        ++issued;
        onward();
        look();
    };
    a.live = true;
    a.n = cursor_take(a.c);
    a.len = source_len(a.c.b);
    look();
    for (int s = 0; s < C::kStages; ++s) issue();

    const float scale2 = p.scale * kLog2e;
    const float cap2 = p.soft_cap * kLog2e, to_cap = p.soft_cap > 0.f ? kLn2 / p.soft_cap : 0.f;
    uint32_t used = 0;
    for (;;) {
        const int n = cursor_take(c);
        const int len = source_len(c.b);
        // ---- the query rows, as fragments of the permuted contraction
        uint32_t qa[KS][4];
        float qs[2] = {0.f, 0.f};
        int limit[2] = {0, 0};
        bool counts[2] = {false, false};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (r >= RH) {
#pragma unroll
                for (int s = 0; s < KS; ++s) qa[s][1] = qa[s][3] = 0;
                continue;
            }
            const PagedRow row = paged_row(p, part, c, g + 8 * r);
            limit[r] = row.limit;
            counts[r] = row.counts;
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) +
                                     (((size_t)row.b * p.Lq + row.i) * p.Hq + c.h * p.G + row.g) * D;
            uint32_t w[KS][2];
            // the thread's 4 * KS elements: 16 contiguous ones per 16-byte
            // chunk of codes, 8 per chunk of bf16
            constexpr int PER = FP8 ? 16 : 8;
#pragma unroll
            for (int x = 0; x < 4 * KS / PER; ++x)
#pragma unroll
                for (int y = 0; y < PER / 8; ++y) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (row.limit > 0) v = *reinterpret_cast<const uint4 *>(q + (t4 + 4 * x) * PER + y * 8);
                    const int s = (x * PER + y * 8) / 4;
                    w[s][0] = v.x;
                    w[s][1] = v.y;
                    w[s + 1][0] = v.z;
                    w[s + 1][1] = v.w;
                }
            qs[r] = scale2;
            if (FP8) {
                uint32_t top = 0; // largest magnitude, as bf16 bits
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        top = max(top, max(w[s][y] & 0x7fffu, (w[s][y] >> 16) & 0x7fffu));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // exponent of the maximum, kept where 2^-e and 2^e are normal
                const int e = top == 0 ? 0 : min(max((int)(top >> 7) - 127, -120), 120);
                const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
                qs[r] *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        w[s][y] = pack_f16x2(__uint_as_float(w[s][y] << 16) * inv,
                                             __uint_as_float(w[s][y] & 0xffff0000u) * inv);
            }
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                qa[s][r] = w[s][0];
                qa[s][2 + r] = w[s][1];
            }
        }
        float o[OB][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float ev_top = -INFINITY; // E: the largest value exponent of the warp's keys
#pragma unroll
        for (int x = 0; x < OB; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[x][y] = 0.f;
        // keys that every row sees need no mask
        int all = INT_MAX;
#pragma unroll
        for (int r = 0; r < RH; ++r) all = min(all, counts[r] ? limit[r] : INT_MAX);
        all = __reduce_min_sync(0xffffffffu, all);

        for (int t = c.t0; t < c.t0 + n; ++t) {
            const int first = t * kTile + warp * kKeys;
            const int valid = min(len - first, kKeys);
            if (valid <= 0) continue;
            const int st = used % C::kStages;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bars + st, (used / C::kStages) & 1, ctx)) != 0;
            if (!ok) continue;
            ++used;
            const uint32_t kb = ring + st * C::kStageBytes, vb = kb + C::kMatBytes;
            const uint32_t eb = exps + st * C::kExpBytes;
            if (valid < kKeys) {
                // values behind the length: whatever is there, weight 0 must give 0
                for (int x = lane; x < (kKeys - valid) * (C::kRowBytes / 16); x += 32) {
                    const int j = valid + x / (C::kRowBytes / 16), ch = x % (C::kRowBytes / 16);
                    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(chunk_at<FP8>(vb, j, ch)), "r"(0) : "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            // ---- S = Q K^T
            float s[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int j = nb * 8 + key_perm(g);
                s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
                for (int x = 0; x < C::kRowBytes / 64; ++x) {
                    const uint4 v = lds128(chunk_at<FP8>(kb, j, t4 + 4 * x));
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    if (FP8) {
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            mma<FP8, ROWS>(s[nb], qa[4 * x + y], e4m3x2_to_f16x2(w[y] & 0xffffu), e4m3x2_to_f16x2(w[y] >> 16));
                    } else {
                        mma<FP8, ROWS>(s[nb], qa[2 * x], w[0], w[1]);
                        mma<FP8, ROWS>(s[nb], qa[2 * x + 1], w[2], w[3]);
                    }
                }
            }
            // ---- logits in base 2; the row maxima
            float vs[NB][2], top[2] = {-INFINITY, -INFINITY}, ev = -INFINITY;
            const bool masked = first + valid > all || valid < kKeys;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int j = nb * 8 + key_perm(2 * t4 + y);
                    float ks = 1.f;
                    if (FP8) {
                        ks = exp_byte_scale(lds8(eb + j));
                        const uint32_t b = lds8(eb + kKeys + j);
                        vs[nb][y] = exp_byte_scale(b);
                        // bytes behind the length and rows without a value do not count;
                        // 12 keeps 2^(kPBias + 127 - E) finite
                        if (j < valid && b != 255u) ev = fmaxf(ev, fmaxf((float)b, 12.f));
                    }
#pragma unroll
                    for (int r = 0; r < RH; ++r) {
                        float x = s[nb][2 * r + y] * (FP8 ? qs[r] * ks : qs[r]);
                        if (to_cap > 0.f) x = cap2 * tanh_near(x * to_cap);
                        if (masked && !(first + j < limit[r])) x = -INFINITY;
                        s[nb][2 * r + y] = x;
                        top[r] = fmaxf(top[r], x);
                    }
                }
            bool grow = false;
            float m_new[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int r = 0; r < RH; ++r) {
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                m_new[r] = top[r] > m[r] + kLazy ? top[r] : m[r]; // a first maximum is above -inf
                grow |= m_new[r] != m[r];
            }
            float ev_new = ev_top;
            if (FP8) {
                ev = fmaxf(ev, __shfl_xor_sync(0xffffffffu, ev, 1));
                ev = fmaxf(ev, __shfl_xor_sync(0xffffffffu, ev, 2));
                ev_new = fmaxf(ev_top, ev); // keys differ by t4 only: the same in every quad
                grow |= ev_new != ev_top;
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int r = 0; r < RH; ++r) {
                    const float f = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - m_new[r]);
                    l[r] *= f;
                    const float fo = FP8 ? (ev_top == -INFINITY ? 0.f : f * ex2_approx(ev_top - ev_new)) : f;
#pragma unroll
                    for (int x = 0; x < OB; ++x) {
                        o[x][2 * r] *= fo;
                        o[x][2 * r + 1] *= fo;
                    }
                    m[r] = m_new[r];
                }
                ev_top = ev_new;
            }
            // 2^(kPBias - E), applied with the value's own scale
            const float pb = FP8 && ev_top != -INFINITY ? ex2_approx(kPBias + 127.f - ev_top) : 1.f;
            // ---- P, and O += P V, 16 keys at a time
#pragma unroll
            for (int kk = 0; kk < NB / 2; ++kk) {
                uint32_t pa[4] = {0, 0, 0, 0}, pl[4] = {0, 0, 0, 0};
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int r = 0; r < RH; ++r) {
                        const int nb = 2 * kk + hf;
                        const float base = m[r] == -INFINITY ? 0.f : m[r];
                        float e[2];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            e[y] = ex2_approx(s[nb][2 * r + y] - base);
                            l[r] += e[y];
                            // a masked key's scale may be anything
                            if (FP8) e[y] = masked && s[nb][2 * r + y] == -INFINITY ? 0.f : e[y] * (vs[nb][y] * pb);
                        }
                        if (FP8) {
                            pa[2 * hf + r] = pack_f16x2(e[0], e[1]);
                        } else {
                            const uint32_t hi = pack_bf16x2(e[0], e[1]);
                            pa[2 * hf + r] = hi;
                            pl[2 * hf + r] = pack_bf16x2(e[0] - __uint_as_float(hi << 16),
                                                         e[1] - __uint_as_float(hi & 0xffff0000u));
                        }
                    }
                const int j0 = kk * 16 + key_perm(2 * t4), j1 = kk * 16 + key_perm(2 * t4 + 1);
                if (FP8) {
                    uint2 v[4]; // a thread's D / 8 codes of a value
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        v[y] = lds64(chunk_at<FP8>(vb, (y & 1 ? j1 : j0) + (y >> 1) * 8, g >> 1) + (g & 1) * 8);
#pragma unroll
                    for (int w = 0; w < 2; ++w)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t sel = z ? 0x7362u : 0x5140u;
                            const uint32_t x0 = w ? __byte_perm(v[0].y, v[1].y, sel) : __byte_perm(v[0].x, v[1].x, sel);
                            const uint32_t x1 = w ? __byte_perm(v[2].y, v[3].y, sel) : __byte_perm(v[2].x, v[3].x, sel);
                            mma<FP8, ROWS>(o[4 * w + 2 * z], pa, e4m3x2_to_f16x2(x0 & 0xffffu), e4m3x2_to_f16x2(x1 & 0xffffu));
                            mma<FP8, ROWS>(o[4 * w + 2 * z + 1], pa, e4m3x2_to_f16x2(x0 >> 16), e4m3x2_to_f16x2(x1 >> 16));
                        }
                } else {
                    uint4 v[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) v[y] = lds128(chunk_at<FP8>(vb, (y & 1 ? j1 : j0) + (y >> 1) * 8, g));
                    const uint32_t u[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                                              {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
                    for (int w = 0; w < 4; ++w)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t sel = z ? 0x7632u : 0x5410u;
                            const uint32_t b0 = __byte_perm(u[0][w], u[1][w], sel);
                            const uint32_t b1 = __byte_perm(u[2][w], u[3][w], sel);
                            mma<FP8, ROWS>(o[2 * w + z], pa, b0, b1);
                            mma<FP8, ROWS>(o[2 * w + z], pl, b0, b1);
                        }
                }
            }
            __syncwarp(); // every lane has read the stage
            issue();
        }

        // ---- the warps' results of the segment meet in warp 0
        float f[2] = {0.f, 0.f}, mt[2] = {-INFINITY, -INFINITY}, lt[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < RH; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (t4 == 0) stat[warp * 16 + g + 8 * r] = make_float2(m[r], l[r]);
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RH; ++r) {
            float2 x[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                x[w] = stat[w * 16 + g + 8 * r];
                mt[r] = fmaxf(mt[r], x[w].x);
            }
            const float base = mt[r] == -INFINITY ? 0.f : mt[r];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) lt[r] += x[w].y * ex2_approx(x[w].x - base);
            f[r] = ex2_approx(m[r] - base);
            if (FP8) f[r] *= ev_top == -INFINITY ? 0.f : ex2_approx(ev_top - 127.f - kPBias);
        }
#pragma unroll
        for (int r = 0; r < RH; ++r) {
            // a thread's values of a row: O blocks 0 .. OB-1 of columns 2 t4 and 2 t4 + 1
            if (r) __syncthreads(); // warp 0 has read the other half's
            if (warp) {
#pragma unroll
                for (int x = 0; x < OB / 2; ++x)
                    merge[((warp - 1) * (OB / 2) + x) * 32 + lane] =
                        make_float4(o[2 * x][2 * r] * f[r], o[2 * x + 1][2 * r] * f[r], o[2 * x][2 * r + 1] * f[r],
                                    o[2 * x + 1][2 * r + 1] * f[r]);
            }
            __syncthreads();
            if (warp) continue;
            const int in_block = g + 8 * r;
            const PagedRow row = paged_row(p, part, c, in_block);
            float v[2][OB]; // the two columns' runs of OB values
#pragma unroll
            for (int x = 0; x < OB / 2; ++x) {
                float4 z = make_float4(o[2 * x][2 * r] * f[r], o[2 * x + 1][2 * r] * f[r], o[2 * x][2 * r + 1] * f[r],
                                       o[2 * x + 1][2 * r + 1] * f[r]);
#pragma unroll
                for (int w = 0; w < kWarps - 1; ++w) {
                    const float4 y = merge[(w * (OB / 2) + x) * 32 + lane];
                    z.x += y.x, z.y += y.y, z.z += y.z, z.w += y.w;
                }
                v[0][2 * x] = z.x, v[0][2 * x + 1] = z.y, v[1][2 * x] = z.z, v[1][2 * x + 1] = z.w;
            }
            // column n, block x: d = n * 8 + x
            if (stores_whole(part, c, n)) {
                if (!row.counts) continue;
                const int hq = c.h * p.G + row.g;
                float fs = 1.f, lr = lt[r], mr = mt[r];
                if (p.sinks) {
                    const float sink = p.sinks[hq] * kLog2e;
                    mr = fmaxf(mt[r], sink);
                    fs = ex2_approx(mt[r] - mr);
                    lr = lr * fs + ex2_approx(sink - mr);
                }
                const float inv = lr == 0.f ? 0.f : fs / lr;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + (((size_t)row.b * p.Lq + row.i) * p.Hq + hq) * D;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint4 w;
                    w.x = pack_bf16x2(v[y][0] * inv, v[y][1] * inv);
                    w.y = pack_bf16x2(v[y][2] * inv, v[y][3] * inv);
                    w.z = pack_bf16x2(v[y][4] * inv, v[y][5] * inv);
                    w.w = pack_bf16x2(v[y][6] * inv, v[y][7] * inv);
                    *reinterpret_cast<uint4 *>(out + (2 * t4 + y) * 8) = w;
                }
                if (t4 == 0)
                    p.lse[((size_t)row.b * p.Hq + hq) * p.Lq + row.i] = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * kLn2;
            } else if (in_block < part.slot_rows) {
                const size_t at = slot_row(part, c) + in_block;
                float *dst = part.o + at * D;
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < OB; x += 4)
                        *reinterpret_cast<float4 *>(dst + (2 * t4 + y) * 8 + x) =
                            make_float4(v[y][x], v[y][x + 1], v[y][x + 2], v[y][x + 3]);
                if (t4 == 0) *reinterpret_cast<float2 *>(part.ml + at * 2) = make_float2(mt[r], lt[r]);
            }
        }
        if (!cursor_next(p, part, c, n)) break;
        __syncthreads(); // stat and merge are free again
    }
    if (!ok) // copies in flight land before the CTA's shared memory goes
        for (; used < issued; ++used)
            wait_drain(bars + used % C::kStages, (used / C::kStages) & 1, kDrainNs);
    await_previous();
}

template <bool FP8, int ROWS>
cudaError_t go(const PagedProblem &p, const PagedPart &part, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s)
{
    auto kern = paged_few_kernel<FP8, ROWS>;
    static std::atomic<uint64_t> set{0}; // devices whose copy of the kernel has its attribute
    const uint64_t bit = 1ull << p.device;
    if (!(set.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<FP8>::kSmem);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_release);
    }
    return launch_dependent(kern, (unsigned)part.ctas, kWarps * 32, Cfg<FP8>::kSmem, s, k, v, p, part);
}

} // namespace

cudaError_t launch_paged_few(const PagedProblem &p, const PagedPart &part, int cache_dtype, const void *tm_k,
                             const void *tm_v, cudaStream_t s)
{
    const CUtensorMap &k = *static_cast<const CUtensorMap *>(tm_k), &v = *static_cast<const CUtensorMap *>(tm_v);
    const bool few = part.row_block == 8;
    if (cache_dtype == RA_E4M3) return few ? go<true, 8>(p, part, k, v, s) : go<true, 16>(p, part, k, v, s);
    return few ? go<false, 8>(p, part, k, v, s) : go<false, 16>(p, part, k, v, s);
}

} // namespace ra
