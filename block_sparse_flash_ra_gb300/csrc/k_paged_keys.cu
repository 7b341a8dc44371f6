// k_paged_keys.cu -- attention over a paged cache for up to 32 (D = 64: 16)
// query rows per kv head and item: decoding steps, drafts, multi-query heads;
// bf16 queries.  The keys are the M side of the tensor-core products.
//
// With few rows a cached byte is used a few times, so the bound is memory:
// 128 keys of 8 bit are 32 KB, 0.74 us of one SM's share of 6.77 TB/s.  What
// stands beside that is made small:
//   S^T (128 keys x rows) = K (128 x D, shared memory) x Q^T
//   O^T (D x rows)       += V^T (D x 128, the same bytes read MN-major) x P^T
// are tcgen05 products with the cached tile as A, exactly as TMA laid it down:
// cached bytes never pass through registers.  Rows are the N side, where 16
// to 96 columns cost no more than reading A does.  (With the rows as M they
// would be padded to 128; mma.sync.m16n8k16 measured 32 cycles each per
// sub-core, and a kernel on it stopped at 46% of memory speed.)
//
// Measured (e4m3, 8 kv heads of 128, 32 query heads): 64 sequences of 17 to
// 8192 tokens 89 us, 6.1 TB/s, 90% of a copy's rate; bf16, 64 x 8192 tokens
// 306 us, all of it; 32 rows on 8 x 32K bf16 tokens 30 us, 63%, of which some
// 12 us are the launches, the start, the end and the join.  From 24 columns on
// the softmax's issue shows: 20 rows on 64 x 1000-3000 e4m3 tokens 77 us, 52%.
//
// 8-bit caches run kind::f8f6f4 on the codes.  The other operand is split
// into e4m3 terms, each in columns of its own, so that nothing is lost to it:
//   q 2^-e = q1 + q2 / 16 (a bf16's 8 bits are two e4m3 significands; error
//            2^-21 of the row's maximum), and the key's scale multiplies s;
//   p 2^(e_v - E) = x1 + x2 / 32 + x3 / 1024 out of f16, so that the values'
//            scales ride on p: 2^-11 relative, and 2^-24 of the row's largest
//            contribution p 2^e_v at the least.  That is what the reference of
//            a row follows, not its largest logit: neither a key of great
//            weight and little value nor a loud value without weight pushes
//            the others out of e4m3's range.  (A reference by the logits and
//            the loudest value row lost whole tails of weights below 2^-18 of
//            the largest; it took 1-3% less time.  A fourth term, 2^-29, takes
//            4% more with 20 rows, a largest contribution of 2^6 instead of
//            2^4, 2^-26, 6%: references move more often.)
// 16-bit caches run kind::f16 in bf16, q as it is, p = x1 + x2 (2^-16).
// Logits, maxima, sums and O are fp32.
//
// D = 64: two tokens of a page lie in one row of 128 values, so a tile is the
// same bytes with 256 tokens.  A query row takes two columns, q in one half of
// the 128 and zeros in the other: S of the even tokens and S of the odd ones.
// P^T has the two columns likewise, and O's lanes d < 64 of the even column and
// d >= 64 of the odd one are the two halves of the result; the rest of the
// product is of no use, and free.  (Products of the register-fed kind,
// mma.sync on widened codes, took 126 us where this takes 54: 64 sequences of
// 8192 e4m3 tokens, 4 kv heads, 16 query heads, 75% of memory speed.)
//
//   warps 0-3 of each warpgroup
//              softmax of 8 rows: thread = key = TMEM lane of S^T.  A row's
//              maximum is over all threads, so it is only looked for when some
//              weight or contribution passes the present reference by what the
//              type of P allows (one barrier with an or); O (TMEM lane = d) is
//              rescaled then and only then.
//   one warp   issues the products, S(i + 1) before P(i) V(i)
//   one warp   loads: a lane per page, K and V in rings of their own
// A tile's softmax is a chain of a few hundred instructions in few warps, so
// rows are spread over warpgroups (8 each) to keep it short, and up to 16
// columns of an 8-bit cache run two CTAs per SM, one's chain under the other's
// (64 x 4096 tokens: 89 us, 105 with one; 64 x up to 512: 20 and 26).  With at
// most 144 registers a CTA of the join finds room beside the two, and starts
// while they end (64 x 100 tokens: 12.8 us, 14.5 with 147 registers).
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "ra_paged.cuh"
#include "ra_sched.cuh"

namespace ra {
namespace {

constexpr int kKeys = 128, kD = 128; // rows of a cached tile, values of a row
constexpr int kRT = 8;         // rows of a softmax warpgroup
constexpr float kNone = -3e38f; // the maximum of no logits: finite, so that no difference is a NaN
// 8-bit caches: a row's largest contribution is 2^kPBias at its reference and
// may grow by 2^kGrow, to 2^8, where e4m3 steps by 16; so a term's rest is 2^3
// at most and enters the next term times kRest.
constexpr float kPBias = 4.f, kGrow = 4.f, kRest = 32.f;
constexpr float kMinExp = 12.f; // least E: 2^(127 + kPBias - E) stays finite
constexpr float kLouder = 64.f; // a value row that far above E raises it: 2^(e_v - E) stays finite
// Weights have to stay finite where references follow contributions: a value
// row 2^kQuiet below the loudest (of its warp, and its warp's below the tile's)
// counts as that loud, a logit passes its reference by kPass at most, and
// references fall, while E rises, by 2^40 at most: for E of value rows between
// 2^-18 and 2^22.  So weights are below 2^100.
constexpr float kQuiet = 30.f, kPass = 60.f, kFallFrom = 100.f, kFallTo = 140.f;
// 16-bit caches: what a weight may pass its reference by.  bf16 has fp32's
// range, but O's sums of weights times values need some of it.
constexpr float kPass16 = 16.f;

template <bool FP8, int RP, int D>
struct Cfg {
    static constexpr int kPar = kD / D, kTokens = kKeys * kPar; // tokens of a row, of a tile
    static constexpr int kMat = kKeys * kD * (FP8 ? 1 : 2); // bytes of a K or V tile
    static constexpr int kHalves = FP8 ? 1 : 2;             // 128-byte wide blocks of a tile
    static constexpr int kGroups = RP / kRT, kSoftThreads = 128 * kGroups, kThreads = kSoftThreads + 64;
    static constexpr int kMmaWarp = 4 * kGroups, kLoadWarp = kMmaWarp + 1;
    static constexpr int kCtasPerSm = FP8 && RP <= 16 ? 2 : 1;
    static constexpr int kStages = FP8 ? (RP == 8 ? 3 : RP == 16 ? 2 : 5) : 3;
    static constexpr int kVStages = FP8 ? (RP > 16 ? 5 : 3) : RP > 16 ? 2 : 3;
    static constexpr int kQTerms = FP8 ? 2 : 1, kPTerms = FP8 ? 3 : 2;
    static constexpr int kNS = (RP * kQTerms + 15) / 16 * 16;             // columns of S^T
    static constexpr int kNO = (RP * kPTerms + 15) / 16 * 16;             // columns of O^T
    static constexpr int kQBytes = kNS * kD * (FP8 ? 1 : 2);
    static constexpr int kPBytes = kNO * kKeys * (FP8 ? 1 : 2);
    static constexpr int kPChunk = kKeys * 16; // 16 bytes of every key: 16 or 8 columns of P^T
    static constexpr int kKOff = 0;
    static constexpr int kVOff = kKOff + kStages * kMat;
    static constexpr int kQOff = kVOff + kVStages * kMat;
    static constexpr int kPOff = kQOff + 2 * kQBytes; // Q of the present and of the next segment
    static constexpr int kExpOff = kPOff + 2 * kPBytes; // per V stage: scale bytes of K, of V
    static constexpr int kRowOff = kExpOff + (FP8 ? kVStages * 2 * kTokens : 0);
    // per row of both segments: place of its output and of its lse (two words each), logit scale, keys it sees;
    // then its factor
    static constexpr int kRowBytes = RP * 24;
    static constexpr int kRedOff = kRowOff + 2 * kRowBytes + RP * 4;
    static constexpr int kOddOff = kRedOff + 4 * kGroups * (kRT + 4) * 4; // O of odd tokens, where rows are pairs
    static constexpr int kBarOff = kOddOff + (kPar == 2 ? RP / 2 * D * 4 : 0);
    static constexpr int kNumBars = 2 * kStages + 3 * kVStages + 2 + 2 + 2 + 2 + 2 + 1;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kSmem = kMiscOff + 16 + 1024;
    static constexpr uint32_t kColO = 2 * kNS;
    static constexpr uint32_t kCols = kColO + kNO <= 64 ? 64 : kColO + kNO <= 128 ? 128 : 256;
    static constexpr uint32_t kIdescS = ((FP8 ? 0u : (1u << 7) | (1u << 10)) | (1u << 4)) |
                                        ((uint32_t)(kNS >> 3) << 17) | ((uint32_t)(kKeys >> 4) << 24);
    // both operands of O^T are MN-major
    static constexpr uint32_t kIdescO = ((FP8 ? 0u : (1u << 7) | (1u << 10)) | (1u << 4)) | (1u << 15) | (1u << 16) |
                                        ((uint32_t)(kNO >> 3) << 17) | ((uint32_t)(kD >> 4) << 24);
    static_assert(kSmem <= (kCtasPerSm == 2 ? 113 : 227) * 1024, "shared memory");
    static_assert(kRedOff % 16 == 0 && (kRT + 4) % 4 == 0, "words of a warp are read by fours");
    static_assert(kBarOff % 8 == 0 && kRowOff % 8 == 0 && kPOff % 1024 == 0 && kExpOff % 128 == 0, "layout");
};

struct Bars {
    uint64_t *k_full, *k_empty, *v_full, *v_empty, *e_full, *s_full, *s_empty, *p_full, *pv_done, *q_full, *drain;
};

template <class C>
__device__ __forceinline__ Bars carve(uint8_t *smem)
{
    Bars b;
    b.k_full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    b.k_empty = b.k_full + C::kStages;
    b.v_full = b.k_empty + C::kStages;
    b.v_empty = b.v_full + C::kVStages;
    b.e_full = b.v_empty + C::kVStages;
    b.s_full = b.e_full + C::kVStages;
    b.s_empty = b.s_full + 2;
    b.p_full = b.s_empty + 2;
    b.pv_done = b.p_full + 2;
    b.q_full = b.pv_done + 2;
    b.drain = b.q_full + 2; // q_full by segment parity
    return b;
}

// Descriptor of an MN-major operand without swizzle: 16 bytes along MN of 8
// K-rows lie together (128 bytes); `chunk` bytes on, the next 16 along MN;
// `k8` bytes on, the next 8 K-rows.
__device__ __forceinline__ uint64_t sdesc_plain_mn(uint32_t saddr, uint32_t chunk, uint32_t k8)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((k8 >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((chunk >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46;
}

// One product step by the whole warp (an elected lane issues).
template <bool FP8>
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if (FP8)
        asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        mma_ss_w(d, a, b, idesc, accumulate);
}

__device__ __forceinline__ void tmem_ld8(uint32_t addr, float *v)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// The softmax warps' own barriers: 1 of all N threads, 2 + g of warpgroup g.
// All pass them the same number of times whatever happens, so they need no
// time limit.
template <int N>
__device__ __forceinline__ void soft_sync()
{
    asm volatile("barrier.sync 1, %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void group_sync(int bar) { asm volatile("barrier.sync %0, 128;" ::"r"(bar) : "memory"); }
__device__ __forceinline__ bool group_or(int bar, bool x)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "barrier.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)x), "r"(bar)
                 : "memory");
    return r != 0;
}

// The largest of a warp's values (NaN does not count).
__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// e4m3x2 codes of two halves, and two halves back from codes
__device__ __forceinline__ uint32_t to_codes(__half2 x)
{
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f16x2 h, %1;\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(r)
        : "r"(*reinterpret_cast<uint32_t *>(&x)));
    return r;
}
__device__ __forceinline__ __half2 from_codes(uint32_t c)
{
    const uint32_t r = e4m3x2_to_f16x2(c);
    return *reinterpret_cast<const __half2 *>(&r);
}

// Offset of 16-byte chunk c of row j in a tile.
__device__ __forceinline__ uint32_t tile_chunk(int j, int c)
{
    return (c >> 3) * (kKeys * 128) + j * 128 + (((c & 7) ^ (j & 7)) << 4);
}

template <bool FP8, int RP, int D>
__global__ void __launch_bounds__(Cfg<FP8, RP, D>::kThreads, Cfg<FP8, RP, D>::kCtasPerSm)
    paged_keys_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      PagedProblem p, PagedPart part)
{
    using C = Cfg<FP8, RP, D>;
    constexpr int kPar = C::kPar, kTokens = C::kTokens;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Bars bars = carve<C>(smem);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kMiscOff + 4);
    const WaitCtx ctx{abort_flag, p.status, p.timeout_ns};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bars.k_full + s, 1);
            mbar_init(bars.k_empty + s, 1);
        }
        for (int s = 0; s < C::kVStages; ++s) {
            mbar_init(bars.v_full + s, 1);
            mbar_init(bars.v_empty + s, 1);
            mbar_init(bars.e_full + s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bars.s_full + s, FP8 ? 2 : 1);
            mbar_init(bars.s_empty + s, C::kSoftThreads);
            mbar_init(bars.p_full + s, C::kSoftThreads);
            mbar_init(bars.pv_done + s, 1);
            mbar_init(bars.q_full + s, C::kSoftThreads);
        }
        mbar_init(bars.drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::kMmaWarp) {
        tmem_alloc(tmem_holder, C::kCols);
        tmem_relinquish();
    }
    if (warp == C::kLoadWarp && lane == 0) {
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

    if (any && warp == C::kLoadWarp) {
        // ------------------------------------------------------------ loads
        // lane x fetches box x of a tile: its page number, then its K and V
        const int box = min(p.c.page, kTokens) / kPar, per = kKeys / box; // rows
        uint32_t i = 0;
        bool ok = true;
        auto entry = [&](int tile, int len) {
            const int first = tile * kTokens + lane * box * kPar;
            return lane < per && first < len ? page_entry(p, part, c.b, first) : 0;
        };
        for (;;) {
            const int n = cursor_take(c), len = source_len(c.b);
            int next = entry(c.t0, len);
            for (int t = c.t0; ok && t < c.t0 + n; ++t, ++i) {
                const int page = next, first = t * kTokens;
                const int boxes = max(0, (min(len - first, kTokens) + box * kPar - 1) / (box * kPar));
                if (t + 1 < c.t0 + n) next = entry(t + 1, len);
                const bool mine = lane < boxes;
                const bool good = mine && page_valid(p, page);
                const int z = good ? page * p.c.Hkv + c.h : p.c.n_pages * p.c.Hkv; // out of range: zeros
                const int off = ((first + lane * box * kPar) & (p.c.page - 1)) / kPar;
                const int sv = i % C::kVStages, sk = i % C::kStages;
                if (!(ok = wait_all(bars.k_empty + sk, ((i / C::kStages) & 1) ^ 1))) break;
                if (lane == 0) mbar_expect_tx(bars.k_full + sk, boxes * box * (C::kMat / kKeys));
                __syncwarp();
                uint8_t *kd = smem + C::kKOff + sk * C::kMat + lane * box * 128;
                if (mine)
                    for (int hf = 0; hf < C::kHalves; ++hf)
                        tma_load_3d(kd + hf * (kKeys * 128), &tm_k, bars.k_full + sk, hf * 64, off, z);
                if (!(ok = wait_all(bars.v_empty + sv, ((i / C::kVStages) & 1) ^ 1))) {
                    ++i; // this tile's K is on its way, its V is not
                    break;
                }
                const int n_good = __popc(__ballot_sync(0xffffffffu, good));
                if (FP8) {
                    uint8_t *e = smem + C::kExpOff + sv * 2 * kTokens + lane * box * kPar;
                    if (mine && !good) { // zeros, at a scale of one
                        for (int j = 0; j < box * kPar; ++j) e[j] = e[kTokens + j] = 127;
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    __syncwarp();
                    if (lane == 0) mbar_expect_tx(bars.e_full + sv, 2 * n_good * box * kPar);
                    __syncwarp();
                    if (good) {
                        const size_t row = ((size_t)z << p.c.page_shift) + off * kPar;
                        bulk_load(e, p.c.k_exp + row, box * kPar, bars.e_full + sv);
                        bulk_load(e + kTokens, p.c.v_exp + row, box * kPar, bars.e_full + sv);
                    }
                }
                if (lane == 0) mbar_expect_tx(bars.v_full + sv, boxes * box * (C::kMat / kKeys));
                __syncwarp();
                uint8_t *vd = smem + C::kVOff + sv * C::kMat + lane * box * 128;
                if (mine)
                    for (int hf = 0; hf < C::kHalves; ++hf)
                        tma_load_3d(vd + hf * (kKeys * 128), &tm_v, bars.v_full + sv, hf * 64, off, z);
            }
            if (!ok || !cursor_next(p, part, c, n)) break;
        }
        if (!ok) {
            // copies on their way land before the CTA ends: tile j's phase of
            // its stage, for the last tiles of each ring (a phase that already
            // passed, or the V that was not asked for, only runs the clock)
            for (uint32_t j = i > (uint32_t)C::kStages ? i - C::kStages : 0; j < i; ++j)
                wait_drain(bars.k_full + j % C::kStages, (j / C::kStages) & 1, kDrainNs);
            for (uint32_t j = i > (uint32_t)C::kVStages ? i - C::kVStages : 0; j < i; ++j) {
                wait_drain(bars.v_full + j % C::kVStages, (j / C::kVStages) & 1, kDrainNs);
                if (FP8) wait_drain(bars.e_full + j % C::kVStages, (j / C::kVStages) & 1, kDrainNs);
            }
        }
    } else if (any && warp == C::kMmaWarp) {
        // ------------------------------------------------------------ products
        const uint64_t kd0 = sdesc_sw128(smem_u32(smem + C::kKOff), 16, 1024);
        const uint64_t vd0 = sdesc_sw128(smem_u32(smem + C::kVOff), kKeys * 128, 1024);
        const uint64_t qd0 = sdesc_sw128(smem_u32(smem + C::kQOff), 16, 1024);
        const uint64_t pd0 = sdesc_plain_mn(smem_u32(smem + C::kPOff), C::kPChunk, 128);
        uint32_t i = 0, segs = 0;
        bool ok = true;
        auto issue_pv = [&](uint32_t j, bool first) -> bool {
            const int sb = j & 1, sv = j % C::kVStages;
            if (!wait_all(bars.v_full + sv, (j / C::kVStages) & 1)) return false;
            if (!wait_all(bars.p_full + sb, (j >> 1) & 1)) return false;
            tc_fence_after();
            const uint64_t vd = vd0 + (uint32_t)((sv * C::kMat) >> 4), pd = pd0 + (uint32_t)((sb * C::kPBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < (FP8 ? 4 : 8); ++kk) {
                // 32 or 16 keys further down both tiles
                const uint32_t bo = kk * (FP8 ? 32 : 16) * 16;
                mma_step<FP8>(tmem + C::kColO, vd + (uint32_t)((kk * (FP8 ? 4096 : 2048)) >> 4), pd + (bo >> 4), C::kIdescO,
                              (kk > 0 || !first) ? 1u : 0u);
            }
            tc_commit_w(bars.v_empty + sv);
            tc_commit_w(bars.pv_done + sb);
            return true;
        };
        for (;;) {
            const int n = cursor_take(c), len = kPar == 2 ? source_len(c.b) : 0;
            if (!(ok = wait_all(bars.q_full + (segs & 1), (segs >> 1) & 1))) break;
            const uint64_t qd = qd0 + (uint32_t)(((segs++ & 1) * C::kQBytes) >> 4);
            for (int t = 0; ok && t < n; ++t, ++i) {
                const int sk = i % C::kStages, sb = i & 1;
                if (!(ok = wait_all(bars.k_full + sk, (i / C::kStages) & 1))) break;
                if (FP8 && !(ok = wait_all(bars.e_full + i % C::kVStages, (i / C::kVStages) & 1))) break;
                if (!(ok = wait_all(bars.s_empty + sb, ((i >> 1) & 1) ^ 1))) break;
                tc_fence_after();
                if (kPar == 2) {
                    // an odd length ends inside a row: its other token meets the zeros of
                    // Q, and is made zero too, whatever is there
                    const int valid = len - (c.t0 + t) * kTokens, j = valid >> 1;
                    if (valid > 0 && valid < kTokens && (valid & 1)) {
                        if (lane < C::kHalves * 4)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                                             smem_u32(smem + C::kKOff + sk * C::kMat) + tile_chunk(j, C::kHalves * 4 + lane)),
                                         "r"(0)
                                         : "memory");
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                }
                const uint64_t kd = kd0 + (uint32_t)((sk * C::kMat) >> 4);
#pragma unroll
                for (int kk = 0; kk < (FP8 ? 4 : 8); ++kk) {
                    const uint32_t ao = FP8 ? kk * 32 : (kk >> 2) * (kKeys * 128) + (kk & 3) * 32;
                    const uint32_t bo = FP8 ? kk * 32 : (kk >> 2) * (C::kNS * 128) + (kk & 3) * 32;
                    mma_step<FP8>(tmem + sb * C::kNS, kd + (ao >> 4), qd + (bo >> 4), C::kIdescS, kk > 0 ? 1u : 0u);
                }
                tc_commit_w(bars.k_empty + sk);
                // the softmax reads the tile's scale bytes as well as S: this arrival
                // passes on what the wait for them has seen
                if (FP8 && lane == 0) mbar_arrive(bars.s_full + sb);
                tc_commit_w(bars.s_full + sb);
                if (t > 0) ok = issue_pv(i - 1, t == 1);
            }
            if (!ok || !(ok = issue_pv(i - 1, n == 1))) break;
            if (!cursor_next(p, part, c, n)) break;
        }
        tc_commit_w(bars.drain);
        wait_drain(bars.drain, 0, kDrainNs);
    } else if (any) {
        // ------------------------------------------------------------ softmax
        // From the first wait that gave up on, a thread makes no wait any more
        // and runs its loops out on whatever is there: every barrier of these
        // warps is still met by all of them, converged.
        constexpr int NT = C::kSoftThreads, RS = kRT + 4; // words of a warp in red
        const int tid = threadIdx.x & 127, grp = threadIdx.x >> 7, row0 = grp * kRT, wq = warp & 3, bar = 2 + grp;
        const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
        float *row_f = reinterpret_cast<float *>(smem + C::kRowOff + 2 * C::kRowBytes);
        float *red = reinterpret_cast<float *>(smem + C::kRedOff) + grp * 4 * RS; // [4 warps][RS]
        const uint32_t p_base = smem_u32(smem + C::kPOff);
        const float cap2 = p.soft_cap * kLog2e, to_cap = p.soft_cap > 0.f ? kLn2 / p.soft_cap : 0.f;
        uint32_t i = 0;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = mbar_wait(bar, parity, ctx);
            __syncwarp();
        };
        // what is known of the rows of segment number `par`
        struct Rows {
            long long *place, *lse; // (b * Lq + i) * Hq + hq, or -1; where its lse goes
            float *qs;
            int *limit;
        };
        auto rows_of = [&](uint32_t par) {
            Rows r;
            r.place = reinterpret_cast<long long *>(smem + C::kRowOff + (par & 1) * C::kRowBytes);
            r.lse = r.place + RP;
            r.qs = reinterpret_cast<float *>(r.lse + RP);
            r.limit = reinterpret_cast<int *>(r.qs + RP);
            return r;
        };
        // Q of the segment at `at`, number `par` of the CTA: 16 threads take a
        // row, 8 values each.  It is fetched a segment ahead; the segment before
        // last, whose place it takes, has all its S behind it.
        auto load_q = [&](const PagedCursor &at, uint32_t par) {
            const Rows ri = rows_of(par);
            const uint32_t q_base = smem_u32(smem + C::kQOff + (par & 1) * C::kQBytes);
#pragma unroll 1
            for (int r = threadIdx.x >> 4; r < C::kNS / C::kQTerms; r += NT / 16) {
                const int x = threadIdx.x & 15;
                const PagedRow row = paged_row(p, part, at, r / kPar);
                const bool live = r < RP && row.counts;
                const int hq = at.h * p.G + row.g;
                const long long place = ((long long)row.b * p.Lq + row.i) * p.Hq + hq;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (live && (kPar == 1 || (x >> 3) == (r & 1)))
                    w = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + (size_t)place * D + (x & (D / 8 - 1)) * 8);
                float qs = p.scale * kLog2e;
                if (FP8) {
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                    uint32_t top = 0; // largest magnitude, as bf16 bits
#pragma unroll
                    for (int y = 0; y < 4; ++y) top = max(top, max(u[y] & 0x7fffu, (u[y] >> 16) & 0x7fffu));
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // the maximum goes to [128, 256); 2^+-e stay normal
                    const int e = min(max((int)(top >> 7) - 134, -120), 120);
                    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
                    qs *= __uint_as_float((uint32_t)(127 + e) << 23);
                    if (top >= 0x7f80u) qs = __uint_as_float(0x7fc00000u); // e4m3 has no infinity
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        // f16 holds the 8 bits; below 2^-14 it rounds at 2^-25
                        const __half2 q2 = __floats2half2_rn(__uint_as_float(u[y] << 16) * inv,
                                                             __uint_as_float(u[y] & 0xffff0000u) * inv);
                        hi[y] = to_codes(q2);
                        lo[y] = to_codes(__hmul2(__hsub2(q2, from_codes(hi[y])), __float2half2_rn(16.f)));
                    }
                    const uint32_t dst = q_base + (((x >> 1) ^ (r & 7)) << 4) + (x & 1) * 8;
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst + r * 128), "r"(hi[0] | hi[1] << 16),
                                 "r"(hi[2] | hi[3] << 16)
                                 : "memory");
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst + (RP + r) * 128), "r"(lo[0] | lo[1] << 16),
                                 "r"(lo[2] | lo[3] << 16)
                                 : "memory");
                } else {
                    const uint32_t dst = q_base + (x >> 3) * (C::kNS * 128) + r * 128 +
                                        (((x & 7) ^ (r & 7)) << 4);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                                 : "memory");
                }
                if (x == 0 && r < RP) {
                    ri.qs[r] = qs;
                    ri.limit[r] = live ? row.limit : 0x7fffffff; // rows of no use need no mask
                    ri.place[r] = live ? place : -1;
                    ri.lse[r] = ((long long)row.b * p.Hq + hq) * p.Lq + row.i;
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(bars.q_full + (par & 1));
        };
        load_q(c, 0);
        for (uint32_t seg = 0;; ++seg) {
            const int n = cursor_take(c), len = source_len(c.b);
            PagedCursor next = c;
            const bool more = cursor_next(p, part, next, n);
            if (more) load_q(next, seg + 1);
            const Rows rows = rows_of(seg);
            soft_sync<NT>();
            float qs[kRT];
            int all = len; // keys below it are seen by every row
#pragma unroll
            for (int r = 0; r < kRT; ++r) {
                qs[r] = rows.qs[row0 + r];
                all = min(all, rows.limit[row0 + r]);
            }

            float m[kRT], l[kRT], ev_top = kMinExp; // references, sums, E
#pragma unroll
            for (int r = 0; r < kRT; ++r) m[r] = kNone, l[r] = 0.f;
            for (int t = c.t0; t < c.t0 + n; ++t, ++i) {
                const int sb = i & 1, sv = i % C::kVStages;
                const int tok = tid * kPar, first = t * kTokens; // the row's first token in the tile
                const int valid = min(len - first, kTokens);
                const bool masked = first + kTokens > all;
                float s[kRT];
                float ks[kPar] = {}, vs[kPar] = {}, ev[kPar] = {};
                wait(bars.s_full + sb, (i >> 1) & 1);
                tc_fence_after();
                tmem_ld8(lane_base + sb * C::kNS + row0, s);
                if (FP8) {
                    const uint8_t *e = smem + C::kExpOff + sv * 2 * kTokens + tok;
#pragma unroll
                    for (int y = 0; y < kPar; ++y) {
                        const uint32_t vb = e[kTokens + y];
                        ks[y] = exp_byte_scale(e[y]);
                        vs[y] = exp_byte_scale(vb);
                        // bytes behind the length and rows without a value do not count
                        ev[y] = tok + y < valid && vb != 255u ? fmaxf((float)vb, kMinExp) : kMinExp;
                    }
                }
                if (FP8) {
                    float s2[kRT];
                    tmem_ld8(lane_base + sb * C::kNS + RP + row0, s2);
                    tmem_ld_wait();
#pragma unroll
                    for (int r = 0; r < kRT; ++r) s[r] = fmaf(s2[r], 1.f / 16.f, s[r]);
                } else {
                    tmem_ld_wait();
                }
                tc_fence_before();
                mbar_arrive(bars.s_empty + sb);
                // ---- logits in base 2
                bool grow = FP8 && fmaxf(ev[0], ev[kPar - 1]) > ev_top + kLouder;
#pragma unroll
                for (int r = 0; r < kRT; ++r) s[r] *= FP8 ? qs[r] * ks[r % kPar] : qs[r];
                if (to_cap > 0.f) {
                    float xa = 0.f;
#pragma unroll
                    for (int r = 0; r < kRT; ++r) xa = fmaxf(xa, fabsf(s[r]));
                    if (__all_sync(0xffffffffu, xa * to_cap < kTanhSmall)) {
#pragma unroll
                        for (int r = 0; r < kRT; ++r) s[r] = cap2 * tanh_series(s[r] * to_cap);
                    } else {
#pragma unroll
                        for (int r = 0; r < kRT; ++r) s[r] = cap2 * tanh_near(s[r] * to_cap);
                    }
                }
                if (masked) {
#pragma unroll
                    for (int r = 0; r < kRT; ++r)
                        if (tok + r % kPar >= valid || first + tok + r % kPar >= rows.limit[row0 + r]) s[r] = -INFINITY;
                }
                // how far a logit may pass its reference: as a weight by kPass or kPass16,
                // as a contribution 2^(s + e_v - E) to an 8-bit cache's O by kGrow.  (Sums are rounded up:
                // a reference must not come out too low.)
                float room[kPar];
#pragma unroll
                for (int y = 0; y < kPar; ++y) room[y] = FP8 ? fmaxf(ev[y] - ev_top - kGrow, -kPass) : -kPass16;
#pragma unroll
                for (int r = 0; r < kRT; ++r) grow |= __fadd_ru(s[r], room[r % kPar]) > m[r];
                if (group_or(bar, grow)) {
                    // new references: the maxima so far
                    float loud = 0.f, quiet[kPar] = {}, top[kRT];
                    if (FP8) {
                        loud = warp_max(fmaxf(ev[0], ev[kPar - 1]));
#pragma unroll
                        for (int y = 0; y < kPar; ++y) quiet[y] = fmaxf(ev[y] - loud, -kQuiet);
                    }
#pragma unroll
                    for (int r = 0; r < kRT; ++r) top[r] = warp_max(FP8 ? __fadd_ru(s[r], quiet[r % kPar]) : s[r]);
                    if (lane == 0) {
                        float4 *mine = reinterpret_cast<float4 *>(red + wq * RS);
                        mine[0] = make_float4(top[0], top[1], top[2], top[3]);
                        mine[1] = make_float4(top[4], top[5], top[6], top[7]);
                        if (FP8) red[wq * RS + kRT] = loud;
                    }
                    // O is still: P V of the tile before has completed
                    if (t > c.t0) wait(bars.pv_done + (sb ^ 1), ((i - 1) >> 1) & 1);
                    group_sync(bar);
                    float fe = 1.f, drop = 0.f;
                    if (FP8) {
                        float e = ev_top;
#pragma unroll
                        for (int w = 0; w < 4; ++w) e = fmaxf(e, red[w * RS + kRT]);
                        drop = fmaxf(fminf(e, kFallTo) - fmaxf(ev_top, kFallFrom), 0.f);
                        fe = ex2_approx(ev_top - e);
                        ev_top = e;
                    }
#pragma unroll
                    for (int r = 0; r < kRT; ++r) top[r] = __fadd_ru(m[r], -drop);
#pragma unroll 2
                    for (int w = 0; w < 4; ++w) { // (all at once would take registers from the join beside)
                        const float4 *of = reinterpret_cast<const float4 *>(red + w * RS), a = of[0], b = of[1];
                        const float x[kRT] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                        const float below = FP8 ? fmaxf(red[w * RS + kRT] - ev_top, -kQuiet) : 0.f;
#pragma unroll
                        for (int r = 0; r < kRT; ++r) top[r] = fmaxf(top[r], __fadd_ru(x[r], below));
                    }
                    float f[kRT];
#pragma unroll
                    for (int r = 0; r < kRT; r += kPar) {
                        const float ref = fmaxf(top[r], top[r + kPar - 1]), x = ex2_approx(m[r] - ref);
#pragma unroll
                        for (int y = 0; y < kPar; ++y) {
                            l[r + y] *= x;
                            f[r + y] = x * fe;
                            m[r + y] = ref;
                        }
                    }
                    if (t > c.t0) {
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < C::kPTerms; ++k) {
                            float o[8];
                            uint32_t w[8];
                            tmem_ld8(lane_base + C::kColO + k * RP + row0, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int y = 0; y < 8; ++y) w[y] = __float_as_uint(o[y] * f[y]);
                            tmem_st8(lane_base + C::kColO + k * RP + row0, w);
                        }
                        tmem_st_wait();
                        tc_fence_before(); // O is written before p_full lets the next P V at it
                    }
                    group_sync(bar); // red is free again
                }
                // ---- weights, as the terms of P^T: column of term k and query row
                // r is k * RP + r, this thread's row is its key.  S of this tile was
                // issued after P V of the tile before last, so that tile's weights
                // have been read.
                const float pb = FP8 ? ex2_approx(127.f + kPBias - ev_top) : 1.f;
                float x[kRT];
#pragma unroll
                for (int r = 0; r < kRT; ++r) {
                    x[r] = ex2_approx(s[r] - m[r]);
                    l[r] += x[r];
                    if (FP8) x[r] *= pb * vs[r % kPar];
                }
                if (FP8 && masked) {
                    // a masked key's scale may be anything
#pragma unroll
                    for (int r = 0; r < kRT; ++r)
                        if (s[r] == -INFINITY) x[r] = 0.f;
                }
                const uint32_t pt = p_base + sb * C::kPBytes + tid * 16;
                if (FP8) {
                    __half2 h[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) h[y] = __floats2half2_rn(x[2 * y], x[2 * y + 1]);
#pragma unroll
                    for (int k = 0; k < C::kPTerms; ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            w[y] = to_codes(h[y]);
                            if (k + 1 < C::kPTerms) h[y] = __hmul2(__hsub2(h[y], from_codes(w[y])), __float2half2_rn(kRest));
                        }
                        const int col = k * RP + row0; // 8 columns: half of a 16-byte chunk
                        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(pt + (col >> 4) * C::kPChunk + (col & 8)),
                                     "r"(__byte_perm(w[0], w[1], 0x5410)), "r"(__byte_perm(w[2], w[3], 0x5410))
                                     : "memory");
                    }
                } else {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        hi[y] = pack_bf16x2(x[2 * y], x[2 * y + 1]);
                        lo[y] = pack_bf16x2(x[2 * y] - __uint_as_float(hi[y] << 16), x[2 * y + 1] - __uint_as_float(hi[y] & 0xffff0000u));
                    }
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(pt + (row0 >> 3) * C::kPChunk), "r"(hi[0]),
                                 "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
                                 : "memory");
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(pt + ((RP + row0) >> 3) * C::kPChunk), "r"(lo[0]),
                                 "r"(lo[1]), "r"(lo[2]), "r"(lo[3])
                                 : "memory");
                }
                if (valid < kTokens) {
                    // values behind the length: whatever is there, weight 0 must give 0
                    wait(bars.v_full + sv, (i / C::kVStages) & 1);
                    if (grp == 0 && tok + kPar > valid)
#pragma unroll 1
                        for (int x = tok < valid ? C::kHalves * 4 : 0; x < C::kHalves * 8; ++x)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                                             smem_u32(smem + C::kVOff + sv * C::kMat) + tile_chunk(tid, x)),
                                         "r"(0)
                                         : "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(bars.p_full + sb);
            }
            // ---- the segment's end: sums over the keys' threads
            // (each step a lane hands half of its rows over: short code, and every
            // lane busy)
#pragma unroll
            for (int h = kRT / 2, w = 16; h; h >>= 1, w >>= 1) {
                const bool up = (lane & w) != 0;
#pragma unroll
                for (int r = 0; r < h; ++r) {
                    const float x = up ? l[r] : l[r + h];
                    l[r] = (up ? l[r + h] : l[r]) + __shfl_xor_sync(0xffffffffu, x, w);
                }
            }
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], 2);
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
            if ((lane & 3) == 0) red[wq * RS + (lane >> 2)] = l[0];
            if (tid == 0) {
                float4 *f4 = reinterpret_cast<float4 *>(row_f + row0);
                f4[0] = make_float4(m[0], m[1], m[2], m[3]);
                f4[1] = make_float4(m[4], m[5], m[6], m[7]);
            }
            soft_sync<NT>();
            const bool final = stores_whole(part, c, n);
            const size_t slot = slot_row(part, c) + row0 / kPar;
            if (tid < kRT / kPar) {
                // a thread per query row: its factor, and what is stored beside O
                const int col = row0 + tid * kPar;
                const long long place = rows.place[col];
                float lr = 0.f, mr = row_f[col], f = 1.f;
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int y = 0; y < kPar; ++y) lr += red[w * RS + tid * kPar + y];
                if (final) {
                    if (p.sinks && place >= 0) {
                        const float sink = p.sinks[place % p.Hq] * kLog2e, top = fmaxf(mr, sink);
                        f = ex2_approx(mr - top);
                        lr = lr * f + ex2_approx(sink - top);
                        mr = top;
                    }
                    f = lr == 0.f ? 0.f : f / lr;
                    if (place >= 0) p.lse[rows.lse[col]] = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * kLn2;
                } else if (place >= 0) {
                    *reinterpret_cast<float2 *>(part.ml + (slot + tid) * 2) = make_float2(mr, lr);
                }
                if (FP8) f *= ex2_approx(ev_top - 127.f - kPBias);
                row_f[col] = f;
            }
            wait(bars.pv_done + ((i - 1) & 1), ((i - 1) >> 1) & 1);
            soft_sync<NT>();
            tc_fence_after();
            float o[C::kPTerms][8];
#pragma unroll
            for (int k = 0; k < C::kPTerms; ++k) tmem_ld8(lane_base + C::kColO + k * RP + row0, o[k]);
            tmem_ld_wait();
            tc_fence_before();
            // a query row's O: this thread's value of it, from all tokens or from
            // those of the thread's parity
            float v[kRT / kPar];
#pragma unroll
            for (int y = 0; y < kRT / kPar; ++y) {
                float z[C::kPTerms];
#pragma unroll
                for (int k = 0; k < C::kPTerms; ++k) z[k] = kPar == 2 && tid >= D ? o[k][y * kPar + kPar - 1] : o[k][y * kPar];
                v[y] = FP8 ? z[0] + (z[1] + z[C::kPTerms - 1] * (1.f / kRest)) * (1.f / kRest) : z[0] + z[1];
                v[y] *= row_f[row0 + y * kPar];
            }
            if (kPar == 2) {
                float *odd = reinterpret_cast<float *>(smem + C::kOddOff) + row0 / kPar * D + (tid & (D - 1));
                if (tid >= D) {
#pragma unroll
                    for (int y = 0; y < kRT / kPar; ++y) odd[y * D] = v[y];
                }
                group_sync(bar);
                if (tid < D) {
#pragma unroll
                    for (int y = 0; y < kRT / kPar; ++y) v[y] += odd[y * D];
                }
            }
#pragma unroll
            for (int y = 0; y < kRT / kPar; ++y) {
                const long long place = rows.place[row0 + y * kPar];
                if (place < 0 || tid >= D) continue;
                if (final) static_cast<__nv_bfloat16 *>(p.out)[(size_t)place * D + tid] = __float2bfloat16_rn(v[y]);
                else part.o[(slot + y) * D + tid] = v[y];
            }
            soft_sync<NT>(); // the rows' arrays and red are free again
            if (!more) break;
            c = next;
        }
    }
    await_previous();
    tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::kCols);
    }
}

template <bool FP8, int RP, int D>
cudaError_t go(const PagedProblem &p, const PagedPart &part, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s)
{
    using C = Cfg<FP8, RP, D>;
    auto kern = paged_keys_kernel<FP8, RP, D>;
    static std::atomic<uint64_t> set{0}; // devices whose copy of the kernel has its attribute
    const uint64_t bit = 1ull << p.device;
    if (!(set.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_release);
    }
    return launch_dependent(kern, (unsigned)part.ctas, C::kThreads, C::kSmem, s, k, v, p, part);
}

} // namespace

cudaError_t launch_paged_keys(const PagedProblem &p, const PagedPart &part, int cache_dtype, const void *tm_k,
                              const void *tm_v, cudaStream_t s)
{
    const CUtensorMap &k = *static_cast<const CUtensorMap *>(tm_k), &v = *static_cast<const CUtensorMap *>(tm_v);
    const int cols = part.row_block * (kD / p.c.D);
    auto typed = [&](auto fp8, auto d) {
        constexpr bool FP8 = decltype(fp8)::value;
        constexpr int D = decltype(d)::value;
        return cols == 8    ? go<FP8, 8, D>(p, part, k, v, s)
               : cols == 16 ? go<FP8, 16, D>(p, part, k, v, s)
               : cols == 24 ? go<FP8, 24, D>(p, part, k, v, s)
                            : go<FP8, 32, D>(p, part, k, v, s);
    };
    auto sized = [&](auto fp8) {
        return p.c.D == 64 ? typed(fp8, std::integral_constant<int, 64>{}) : typed(fp8, std::integral_constant<int, 128>{});
    };
    return cache_dtype == RA_E4M3 ? sized(std::true_type{}) : sized(std::false_type{});
}

} // namespace ra
