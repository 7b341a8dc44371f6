// ra_paged.cuh -- device parts shared by the paged attention kernels: the
// spread of the work over CTAs, the numbering of partial results, and the
// cached rows' scales.
//
// Work.  A source's keys are cut into tiles of `tile` tokens; a segment is the
// run of tiles of one (sequence, row block, kv head).  All segments lie on one
// line -- sequences in order, in each its row blocks, in each its kv heads --
// each as `seg_cost` empty places (what taking up a segment costs, in tiles)
// and then its tiles, and CTA c of C takes the c-th share of ceil(N / C)
// places.  Shares cost about the same whatever the lengths are, and lengths
// stay on the device: every CTA adds up the lengths of the batch itself (B
// integers out of L2) to find where its share begins.  They must not change
// while a call runs, but every loop here ends, and every index stays in
// bounds, if they do.
//
// Partial results.  Where whole segments are stored by the CTA that has them
// (`direct`), a CTA leaves at most two partial results, of the first and the
// last segment of its share: slots 2c and 2c + 1.  Otherwise CTA c's part of
// segment s goes to slot c + s: along the line both numbers only grow, and
// each new (CTA, segment) pair raises at least one of them, so no two pairs
// share a slot, and C + S slots are enough.  The join finds a segment's slots
// from the same sums.
#pragma once

#include "ra_device.cuh"
#include "ra_paged.h"

namespace ra {

// The next kernel of the stream may be placed beside this one.
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// The kernels before this one in the stream have ended (see launch_dependent).
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// An attention kernel's place in the stream.  The sequences' own part reads
// what earlier kernels wrote (lengths, tables, queries, the cache) and reuses
// the workspace, so it waits for them, and only then lets the next kernel in;
// the prefix's part comes behind it, so all of that holds already.
__device__ __forceinline__ void begin_in_order(const PagedPart &part)
{
    if (!part.prefix) await_previous();
    allow_next();
}

__device__ __forceinline__ void report_bad_page(int *status) { atomicMax(status + kBadPageWord, 1); }

// 2^(b - 127) of a cached row's scale byte; 255 marks a row without a value.
// (0, which ra_kv_write does not store, is a subnormal power of two.)
__device__ __forceinline__ float exp_byte_scale(uint32_t b)
{
    return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}

// What a row's logits are taken relative to: their maximum, or 0 where nothing
// is seen (and the sink is -inf), so that no difference is -inf - -inf.
__device__ __forceinline__ float finite_base(float top) { return top == -INFINITY ? 0.f : top; }

// tanh by its series, for |x| < kTanhSmall.
__device__ __forceinline__ float tanh_series(float x)
{
    const float z = x * x;
    return x * fmaf(z, fmaf(z, fmaf(z, kTanhC7, kTanhC5), kTanhC3), 1.f);
}
// For any x.  1 - 2 / (1 + e^2x) is off by some 2^-23 whatever x is: times a
// soft cap of 50 that is 10^-5 of a logit near 1, so small x take the series.
__device__ __forceinline__ float tanh_near(float x)
{
    return fabsf(x) < kTanhSmall ? tanh_series(x) : tanh_fast(x);
}

// Two e4m3 codes (low and high byte of a 16-bit word) as two halves.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ int paged_q_len(const PagedProblem &p, int b)
{
    if (!p.q_len) return p.Lq;
    return min(max(p.q_len[b], 0), p.Lq);
}

__device__ __forceinline__ int paged_kv_len(const PagedProblem &p, int b)
{
    const long long cap = (long long)p.max_pages << p.c.page_shift;
    return (int)min((long long)max(p.kv_len[b], 0), cap);
}

__device__ __forceinline__ int paged_prefix_len(const PagedProblem &p)
{
    const long long cap = (long long)p.prefix_pages << p.c.page_shift;
    return (int)min((long long)max(*p.prefix_len, 0), cap);
}

// Tiles of one segment of sequence b (own keys; 0 when it has no queries).
__device__ __forceinline__ int own_tiles(const PagedProblem &p, const PagedPart &part, int b)
{
    if (paged_q_len(p, b) == 0) return 0;
    return (paged_kv_len(p, b) + part.tile - 1) / part.tile;
}

// Places on the line of one segment of sequence b.
__device__ __forceinline__ int own_places(const PagedProblem &p, const PagedPart &part, int b)
{
    const int n = own_tiles(p, part, b);
    return n ? n + part.seg_cost : 0;
}

// Sums of own_places over all sequences and, in `before`, over those below
// `b_end`; by one converged warp.  (The host refuses problems whose line could
// have 2^31 places.)
__device__ __forceinline__ unsigned own_places_sum(const PagedProblem &p, const PagedPart &part,
                                                   int b_end, unsigned &before)
{
    unsigned n = 0, lo = 0;
#pragma unroll 1
    for (int b = threadIdx.x & 31; b < p.B; b += 32) {
        const int x = own_places(p, part, b);
        n += x;
        if (b < b_end) lo += x;
    }
    before = __reduce_add_sync(0xffffffffu, lo);
    return __reduce_add_sync(0xffffffffu, n);
}

// A place on the line, kept by every thread of a CTA alike.
struct PagedCursor {
    int left;      // places from the next tile on that are the CTA's
    int b, rb, h;  // the segment
    int t0, tiles; // its next tile, and its tiles
    int seg;       // its number
    bool first;    // the first of the share
};

// Places the cursor at CTA `cta`'s first tile.  Called by one converged warp
// (all lanes get the result); false when the share has no tile.
__device__ __forceinline__ bool cursor_begin(const PagedProblem &p, const PagedPart &part, int cta,
                                             PagedCursor &c)
{
    const int per_seq = part.n_rb * p.c.Hkv; // segments of one sequence
    const int lane = threadIdx.x & 31;
    int prefix_tiles = 0;
    unsigned total, before = 0;
    int first32 = 0; // places of one of the first 32 sequences
    if (part.prefix) {
        prefix_tiles = (paged_prefix_len(p) + part.tile - 1) / part.tile;
        total = prefix_tiles ? per_seq * (prefix_tiles + part.seg_cost) : 0;
    } else {
        first32 = lane < p.B ? own_places(p, part, lane) : 0;
        unsigned sum = first32;
#pragma unroll 1
        for (int b = lane + 32; b < p.B; b += 32) sum += own_places(p, part, b);
        total = __reduce_add_sync(0xffffffffu, sum) * per_seq;
    }
    const unsigned share = (total + part.ctas - 1) / part.ctas;
    const unsigned at = share * cta, end = min(at + share, total);
    if (at >= end) return false;
    c.b = 0;
    c.tiles = prefix_tiles;
    if (!part.prefix) {
        // 32 sequences at a time: the first whose running total passes `at`
#pragma unroll 1
        for (int b0 = 0;; b0 += 32) {
            if (b0 >= p.B) return false; // lengths that shrink meanwhile
            const int b = b0 + lane;
            const int n = b0 == 0 ? first32 : b < p.B ? own_places(p, part, b) : 0;
            unsigned run = n * per_seq;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned x = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += x;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + run > at);
            if (past) {
                const int l = __ffs(past) - 1, places = __shfl_sync(0xffffffffu, n, l);
                c.b = b0 + l;
                c.tiles = places - part.seg_cost;
                before += __shfl_sync(0xffffffffu, run, l) - places * per_seq;
                break;
            }
            before += __shfl_sync(0xffffffffu, run, 31);
        }
    }
    const int places = c.tiles + part.seg_cost;
    const int in_seq = (at - before) / (unsigned)places;
    const int off = at - before - in_seq * places;
    c.t0 = max(off - part.seg_cost, 0);
    c.left = (int)(end - at) - max(part.seg_cost - off, 0);
    c.rb = in_seq / p.c.Hkv;
    c.h = in_seq - c.rb * p.c.Hkv;
    c.seg = c.b * per_seq + in_seq;
    c.first = true;
    return c.left > 0;
}

// Tiles of the present segment that fall into the share.
__device__ __forceinline__ int cursor_take(const PagedCursor &c)
{
    return min(c.tiles - c.t0, c.left);
}

// Moves on to the segment after the `n` tiles that cursor_take gave; false at
// the share's end.
__device__ __forceinline__ bool cursor_next(const PagedProblem &p, const PagedPart &part,
                                            PagedCursor &c, int n)
{
    c.left -= n + part.seg_cost;
    if (c.left <= 0) return false;
    c.t0 = 0;
    c.first = false;
    ++c.seg;
    if (++c.h == p.c.Hkv) {
        c.h = 0;
        if (++c.rb == part.n_rb) {
            c.rb = 0;
            do { // a share that goes on has a sequence with tiles ahead
                if (++c.b >= p.B) return false;
                c.tiles = own_tiles(p, part, c.b);
                if (!c.tiles) c.seg += part.n_rb * p.c.Hkv;
            } while (!c.tiles);
        }
    }
    return true;
}

// The first row of the partial result of the present segment.
__device__ __forceinline__ size_t slot_row(const PagedPart &part, const PagedCursor &c)
{
    const size_t slot = part.direct ? 2 * (size_t)blockIdx.x + (c.first ? 0 : 1) : (size_t)blockIdx.x + c.seg;
    return slot * part.slot_rows;
}

// Whether this CTA has the whole segment and stores its rows itself.
__device__ __forceinline__ bool stores_whole(const PagedPart &part, const PagedCursor &c, int n)
{
    return part.direct && c.t0 == 0 && n == c.tiles;
}

// Where query row `row` of an item's row block lies, and which of the
// source's keys it sees: [0, limit), 0 for rows that are not computed.
struct PagedRow {
    int b, i, g, limit;
    bool counts; // a row that is computed (it may see nothing all the same)
};

__device__ __forceinline__ PagedRow paged_row(const PagedProblem &p, const PagedPart &part,
                                              const PagedCursor &c, int row)
{
    PagedRow r;
    const int n = c.rb * part.row_block + row;
    r.b = part.prefix ? n / (p.Lq * p.G) : c.b;
    const int in_seq = part.prefix ? n - r.b * (p.Lq * p.G) : n;
    r.i = in_seq / p.G;
    r.g = in_seq - r.i * p.G;
    r.limit = 0;
    r.counts = false;
    if (n < part.rows) {
        const int qn = paged_q_len(p, r.b);
        if (r.i < qn) {
            r.counts = true;
            if (part.prefix) {
                r.limit = paged_prefix_len(p);
            } else {
                const int len = paged_kv_len(p, r.b);
                r.limit = p.causal ? max(len - qn + r.i + 1, 0) : len;
            }
        }
    }
    return r;
}

// The table's entry for token position t of the item's source.
__device__ __forceinline__ int page_entry(const PagedProblem &p, const PagedPart &part, int b, int t)
{
    const int n = t >> p.c.page_shift;
    return part.prefix ? p.prefix_table[n] : p.page_table[(size_t)b * p.max_pages + n];
}

// Whether an entry names a page of the cache; if not, that is reported.
__device__ __forceinline__ bool page_valid(const PagedProblem &p, int page)
{
    if (page >= 0 && page < p.c.n_pages) return true;
    report_bad_page(p.status);
    return false;
}

// The lengths that had to be clamped are reported once per launch.
__device__ __forceinline__ void report_lengths(const PagedProblem &p, const PagedPart &part)
{
    if (blockIdx.x != 0 || threadIdx.x >= 32) return;
    bool bad = false;
    if (part.prefix) {
        bad = paged_prefix_len(p) != *p.prefix_len;
    } else {
        for (int b = threadIdx.x; b < p.B; b += 32)
            bad |= paged_kv_len(p, b) != p.kv_len[b] || (p.q_len && paged_q_len(p, b) != p.q_len[b]);
    }
    if (bad) report_bad_page(p.status);
}

} // namespace ra
