// ra_paged_api.cu -- the C ABI of the paged cache (include/ra.h): argument
// checks, the choice of kernels and the workspace's layout.
#include <cuda.h>

#include <cstdio>

#include "ra_paged.h"

namespace ra {
namespace {

int refuse(int code, const char *msg) { return set_last_error(code, msg); }

template <typename... A>
int refuse(int code, const char *fmt, A... a)
{
    char msg[256];
    snprintf(msg, sizeof(msg), fmt, a...);
    return set_last_error(code, msg);
}

const char *const kTooLarge = "too many query rows and pages for one call: split the batch";

bool is_aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

int check_cache(const ra_kv_cache *c)
{
    if (!c) return refuse(RA_ERR_INVALID_ARG, "cache is NULL");
    if (c->n_pages <= 0 || c->Hkv <= 0)
        return refuse(RA_ERR_INVALID_ARG, "cache sizes must be positive (n_pages=%d Hkv=%d)", c->n_pages, c->Hkv);
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return refuse(RA_ERR_INVALID_ARG, "page_size must be 16, 32, 64 or 128 (got %d)", c->page_size);
    if (c->D != 64 && c->D != 128) return refuse(RA_ERR_UNSUPPORTED, "D must be 64 or 128 (got %d)", c->D);
    if (c->dtype != RA_BF16 && c->dtype != RA_E4M3)
        return refuse(RA_ERR_INVALID_ARG, "the cache's dtype must be RA_BF16 or RA_E4M3");
    if ((long long)c->n_pages * c->Hkv > 0x7fffffffll)
        return refuse(RA_ERR_UNSUPPORTED, "n_pages * Hkv must be below 2^31");
    if (!c->k || !c->v) return refuse(RA_ERR_INVALID_ARG, "cache tensors are NULL");
    if (!is_aligned(c->k, 16) || !is_aligned(c->v, 16))
        return refuse(RA_ERR_INVALID_ARG, "cache tensors must be 16-byte aligned");
    if (c->dtype == RA_E4M3) {
        if (!c->k_exp || !c->v_exp) return refuse(RA_ERR_INVALID_ARG, "an e4m3 cache needs k_exp and v_exp");
        if (!is_aligned(c->k_exp, 16) || !is_aligned(c->v_exp, 16))
            return refuse(RA_ERR_INVALID_ARG, "k_exp and v_exp must be 16-byte aligned");
    } else if (c->k_exp || c->v_exp) {
        return refuse(RA_ERR_INVALID_ARG, "a bf16 cache has no k_exp and v_exp");
    }
    return RA_OK;
}

int check_dense(int B, int L, int Hkv, int dtype, const int32_t *page_table, int max_pages)
{
    if (B <= 0 || L <= 0 || max_pages <= 0)
        return refuse(RA_ERR_INVALID_ARG, "sizes must be positive (B=%d L=%d max_pages=%d)", B, L, max_pages);
    if (dtype != RA_BF16 && dtype != RA_FP32)
        return refuse(RA_ERR_INVALID_ARG, "dtype must be RA_BF16 or RA_FP32");
    if (!page_table) return refuse(RA_ERR_INVALID_ARG, "page_table is NULL");
    if ((long long)L * Hkv > 0x7fffffffll) return refuse(RA_ERR_UNSUPPORTED, "L * Hkv must be below 2^31");
    return RA_OK;
}

PagedCache cache_of(const ra_kv_cache *c)
{
    PagedCache x{};
    x.k = c->k;
    x.v = c->v;
    x.k_exp = c->k_exp;
    x.v_exp = c->v_exp;
    x.n_pages = c->n_pages;
    x.page = c->page_size;
    x.page_shift = __builtin_ctz((unsigned)c->page_size);
    x.Hkv = c->Hkv;
    x.D = c->D;
    return x;
}

int check_paged(const ra_kv_cache *c, const ra_paged_params *p)
{
    const int rc = check_cache(c);
    if (rc) return rc;
    if (!p) return refuse(RA_ERR_INVALID_ARG, "params is NULL");
    if (p->B <= 0 || p->Lq <= 0 || p->Hq <= 0)
        return refuse(RA_ERR_INVALID_ARG, "sizes must be positive (B=%d Lq=%d Hq=%d)", p->B, p->Lq, p->Hq);
    if (p->Hq % c->Hkv) return refuse(RA_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", p->Hq, c->Hkv);
    if ((double)p->B * p->Lq * p->Hq > 2147483647.0)
        return refuse(RA_ERR_UNSUPPORTED, "B * Lq * Hq must be below 2^31");
    if (p->dtype != RA_BF16 && p->dtype != RA_FP32)
        return refuse(RA_ERR_INVALID_ARG, "dtype must be RA_BF16 or RA_FP32");
    if (!(p->scale > 0.f) || !(p->scale < 1e30f))
        return refuse(RA_ERR_INVALID_ARG, "scale must be positive and finite");
    if (!(p->soft_cap < 1e30f) || (p->soft_cap > 0.f && p->soft_cap < 1e-20f))
        return refuse(RA_ERR_INVALID_ARG, "soft_cap must be finite, and 0 or at least 1e-20");
    if (!p->page_table || !p->kv_len || p->max_pages <= 0)
        return refuse(RA_ERR_INVALID_ARG, "page_table and kv_len are needed, with max_pages > 0");
    if (p->prefix_pages < 0 || (p->prefix_pages > 0) != (p->prefix_table != nullptr) ||
        (p->prefix_pages > 0) != (p->prefix_len != nullptr))
        return refuse(RA_ERR_INVALID_ARG, "prefix_pages, prefix_table and prefix_len must come together");
    if (((long long)p->max_pages + p->prefix_pages) * c->page_size > 0x7fffff00ll) // a tile's end fits too
        return refuse(RA_ERR_UNSUPPORTED, "sequences must be shorter than 2^31 - 256 tokens");
    return RA_OK;
}

// Places on the line of a part's work (ra_paged.cuh) at full tables.
double most_places(const ra_kv_cache *c, const ra_paged_params *p, const PagedPart &a)
{
    const long long tokens = (long long)(a.prefix ? p->prefix_pages : p->max_pages) * c->page_size;
    const long long tiles = (tokens + a.tile - 1) / a.tile + a.seg_cost;
    return (double)tiles * (a.prefix ? 1 : p->B) * a.n_rb * c->Hkv;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// CTAs of one attention launch are a fixed figure, so that the workspace's
// size does not depend on the device (GB300 has 152 SMs).
constexpr int kSms = 152;

enum { kF32, kKeysM, kRowsM };

struct Plan {
    bool fits; // no part is too large
    PagedPart part[2];
    int kernel[2];
    int n_parts;
    size_t bytes; // of the workspace
};

// The kernels of a problem: the sequences' own keys, and the shared prefix.
Plan make_plan(const ra_kv_cache *c, const ra_paged_params *p, uint8_t *ws)
{
    Plan pl{};
    pl.fits = true;
    const int G = p->Hq / c->Hkv;
    for (int k = 0; k < (p->prefix_pages ? 2 : 1); ++k) {
        PagedPart &a = pl.part[pl.n_parts];
        int &kernel = pl.kernel[pl.n_parts++];
        a.prefix = k;
        a.rows = (k ? p->B * p->Lq : p->Lq) * G;
        // seg_cost, in tiles: with the line's shares weighted so, CTAs end
        // together.  Taking up a segment (Q, the first maximum, the results)
        // measured 2.8 us beside tiles of 0.7 us in the keys kernel, and 7 us
        // beside tiles of 1.5 us in the rows kernel.  (16-bit tiles are twice as
        // long, but 2 serves them no better: 128 sequences of 64-1024 tokens 64 us
        // and 58 with 4, 64 of up to 512 30 and 27, 64 of up to 8192 162 and 162.)
        if (p->dtype == RA_FP32) {
            kernel = kF32;
            a.seg_cost = 1;
            a.row_block = a.rows <= 4 ? 4 : 8;
            a.tile = kPagedF32Tile;
            a.ctas = paged_f32_per_sm(a.row_block, c->dtype == RA_E4M3) * kSms;
        } else if (c->D == 128 && a.rows > 32) {
            // against blocks of 32 rows of the keys kernel, 16 sequences of 8192
            // tokens, 4 kv heads: e4m3 40 rows 68 us (keys 72), 64 rows 69 (72),
            // 128 rows 74 (131); bf16 58 (94), 59 (95), 65 (164).  20 rows, 2 x 64K
            // tokens: 44 us (keys 26).
            kernel = kRowsM;
            a.seg_cost = 5;
            a.row_block = 256;
            a.by_groups = 1;
            a.tile = kPagedRowsTile;
            a.ctas = kSms;
        } else {
            kernel = kKeysM;
            a.seg_cost = 4;
            // The narrowest block that holds the rows: 20 rows on 2 x 64K e4m3
            // tokens as one block of 24 24 us, of 32 26, as blocks of 16 28, of 8
            // 30; 32 rows on 8 x 32K bf16 tokens 32 us, in 16s 35, in 8s 52.  At
            // D = 64 more rows go in blocks of 16, too.
            const int par = 128 / c->D; // columns of a query row
            const int cols = a.rows * par >= 32 ? 32 : (a.rows * par + 7) / 8 * 8;
            a.row_block = cols / par;
            a.tile = kPagedKeysTile * par;
            a.ctas = (c->dtype == RA_E4M3 && cols <= 16 ? 2 : 1) * kSms;
        }
        a.n_rb = (a.rows + a.row_block - 1) / a.row_block;
        a.slot_rows = a.rows < a.row_block ? a.rows : a.row_block;
        // places are counted in 32 bits; a CTA without a place has nothing to do
        const double places = most_places(c, p, a);
        pl.fits &= places < 2147483648.0;
        if (places < a.ctas) a.ctas = (int)places;
        a.direct = p->prefix_pages == 0;
        const size_t slots =
            a.direct ? 2 * (size_t)a.ctas : (size_t)a.ctas + (size_t)(k ? 1 : p->B) * a.n_rb * c->Hkv;
        a.o = reinterpret_cast<float *>(ws + pl.bytes);
        pl.bytes += up256(slots * a.slot_rows * c->D * 4);
        a.ml = reinterpret_cast<float *>(ws + pl.bytes);
        pl.bytes += up256(slots * a.slot_rows * 8);
    }
    return pl;
}

} // namespace
} // namespace ra

using namespace ra;

extern "C" {

RA_API int ra_kv_write(const ra_kv_cache *cache, const void *k, const void *v, int dtype, int B, int L,
                       size_t k_stride, size_t v_stride, const int32_t *page_table, int max_pages,
                       const int32_t *start, const int32_t *count, ra_stream_t stream)
{
    int rc = check_cache(cache);
    if (rc || (rc = check_dense(B, L, cache->Hkv, dtype, page_table, max_pages))) return rc;
    if (!k || !v || !start) return refuse(RA_ERR_INVALID_ARG, "k, v and start are needed");
    const size_t row = (size_t)cache->Hkv * cache->D, item = dtype == RA_BF16 ? 2 : 4;
    if (k_stride < row || v_stride < row)
        return refuse(RA_ERR_INVALID_ARG, "strides must be at least Hkv * D (%zu)", row);
    if (!is_aligned(k, 16) || !is_aligned(v, 16) || (k_stride * item) % 16 || (v_stride * item) % 16)
        return refuse(RA_ERR_INVALID_ARG, "k, v and their strides must be 16-byte aligned");
    DeviceInfo d;
    if ((rc = device_info(&d))) return rc;
    const cudaError_t e =
        launch_kv_write(cache_of(cache), cache->dtype, k, v, dtype, B, L, k_stride, v_stride, page_table, max_pages,
                        start, count, d.status, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_cuda_error(e, "kv write launch");
    count_launches(1);
    return RA_OK;
}

RA_API int ra_kv_read(const ra_kv_cache *cache, const int32_t *page_table, int max_pages, const int32_t *kv_len,
                      int B, int L, void *k, void *v, int dtype, ra_stream_t stream)
{
    int rc = check_cache(cache);
    if (rc || (rc = check_dense(B, L, cache->Hkv, dtype, page_table, max_pages))) return rc;
    if (!k || !v || !kv_len) return refuse(RA_ERR_INVALID_ARG, "k, v and kv_len are needed");
    if (!is_aligned(k, 16) || !is_aligned(v, 16)) return refuse(RA_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
    const size_t n = (size_t)B * L * cache->Hkv * cache->D * (dtype == RA_BF16 ? 2 : 4);
    if (overlap(k, n, v, n)) return refuse(RA_ERR_INVALID_ARG, "k and v overlap");
    DeviceInfo d;
    if ((rc = device_info(&d))) return rc;
    const cudaError_t e =
        launch_kv_read(cache_of(cache), cache->dtype, page_table, max_pages, kv_len, B, L, k, v, dtype, d.status,
                       reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_cuda_error(e, "kv read launch");
    count_launches(1);
    return RA_OK;
}

RA_API size_t ra_attn_paged_workspace_size(const ra_kv_cache *cache, const ra_paged_params *p)
{
    if (check_paged(cache, p) != RA_OK) return 0;
    const Plan pl = make_plan(cache, p, nullptr);
    if (!pl.fits) return refuse(RA_ERR_UNSUPPORTED, kTooLarge), 0;
    return pl.bytes;
}

RA_API int ra_attn_paged(const ra_kv_cache *cache, const ra_paged_params *p, const void *q, void *out, float *lse,
                         void *ws, size_t ws_bytes, ra_stream_t stream)
{
    int rc = check_paged(cache, p);
    if (rc) return rc;
    if (!q || !out || !lse) return refuse(RA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!is_aligned(q, 16) || !is_aligned(out, 16) || !is_aligned(lse, 4))
        return refuse(RA_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
    const size_t n = (size_t)p->B * p->Lq * p->Hq * cache->D * (p->dtype == RA_BF16 ? 2 : 4);
    if (overlap(q, n, out, n)) return refuse(RA_ERR_INVALID_ARG, "q and out overlap");
    const Plan pl = make_plan(cache, p, static_cast<uint8_t *>(ws));
    if (!pl.fits) return refuse(RA_ERR_UNSUPPORTED, kTooLarge);
    if (!ws || ws_bytes < pl.bytes)
        return refuse(RA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws ? ws_bytes : (size_t)0, pl.bytes);
    if (!is_aligned(ws, 256)) return refuse(RA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    DeviceInfo d;
    if ((rc = device_info(&d))) return rc;
    PagedProblem x{};
    x.c = cache_of(cache);
    x.B = p->B;
    x.Lq = p->Lq;
    x.Hq = p->Hq;
    x.G = p->Hq / cache->Hkv;
    x.scale = p->scale;
    x.soft_cap = p->soft_cap > 0.f ? p->soft_cap : 0.f;
    x.causal = p->causal ? 1 : 0;
    x.page_table = p->page_table;
    x.max_pages = p->max_pages;
    x.kv_len = p->kv_len;
    x.q_len = p->q_len;
    x.prefix_table = p->prefix_table;
    x.prefix_pages = p->prefix_pages;
    x.prefix_len = p->prefix_len;
    x.sinks = p->sinks;
    x.q = q;
    x.out = out;
    x.lse = lse;
    x.status = d.status;
    x.timeout_ns = d.timeout_ns;
    x.device = d.index;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    for (int k = 0; k < pl.n_parts && e == cudaSuccess; ++k) {
        const PagedPart &part = pl.part[k];
        if (pl.kernel[k] == kF32) {
            e = launch_paged_f32(x, part, cache->dtype, s);
            continue;
        }
        const int most = pl.kernel[k] == kRowsM && cache->dtype == RA_E4M3 ? 64 : 128; // of a box
        const int in_page = cache->page_size * cache->D / 128, rows = in_page < most ? in_page : most;
        CUtensorMap tk, tv;
        if ((rc = encode_paged(&tk, cache, cache->k, rows)) || (rc = encode_paged(&tv, cache, cache->v, rows))) return rc;
        e = pl.kernel[k] == kKeysM ? launch_paged_keys(x, part, cache->dtype, &tk, &tv, s)
                                   : launch_paged_rows(x, part, cache->dtype, &tk, &tv, s);
    }
    if (e == cudaSuccess) e = launch_paged_join(x, pl.part, pl.n_parts, p->dtype, s);
    if (e != cudaSuccess) return set_cuda_error(e, "paged attention launch");
    count_launches(pl.n_parts + 1);
    return RA_OK;
}

} // extern "C"
