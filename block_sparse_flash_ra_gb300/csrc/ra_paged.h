// ra_paged.h -- declarations shared by the paged entry points and kernels.
#pragma once

#include "ra_internal.h"

namespace ra {

// A paged cache in device-friendly form; page sizes are powers of two.
struct PagedCache {
    const void *k, *v;
    const uint8_t *k_exp, *v_exp; // e4m3 only
    int n_pages, page, page_shift, Hkv, D;
};

// One cached-attention problem.  Query rows of one kv head are numbered
// i * G + g inside a sequence, and (b * Lq + i) * G + g over the batch.
struct PagedProblem {
    PagedCache c;
    int B, Lq, Hq, G;
    float scale, soft_cap; // soft_cap 0 = none
    int causal;
    const int32_t *page_table;
    int max_pages;
    const int32_t *kv_len, *q_len;
    const int32_t *prefix_table;
    int prefix_pages;
    const int32_t *prefix_len;
    const float *sinks;
    const void *q;
    void *out;
    float *lse;
    int *status;
    uint64_t timeout_ns;
    int device;
};

// How one launch spreads a source of keys (the sequences' own pages, or the
// shared prefix) over its CTAs; see ra_paged.cuh.
struct PagedPart {
    int prefix;    // 1: the shared prefix, every sequence's rows together
    int rows;      // query rows per kv head of one sequence, or of the batch
    int row_block; // rows of one work item
    int n_rb;      // ceil(rows / row_block)
    int tile;      // keys of one tile
    int ctas;
    int seg_cost;  // what taking up a segment costs, in tiles
    int direct;    // 1: rows whose keys one CTA sees are stored by it
    int slot_rows; // rows that one partial result holds
    int by_groups; // o is (slots, D / 4, slot_rows, 4), not (slots, slot_rows, D)
    float *o;      // unnormalised outputs
    float *ml;     // (slots, slot_rows, 2) row maximum (base-2 logits) and sum
};

// Launches a kernel that may start before its predecessor in the stream has
// ended, once all of that kernel's CTAs have allowed it or are gone.  It
// waits (griddepcontrol.wait) before it touches what came before it, and
// every CTA of an attention kernel waits before it ends, so that its end
// implies the end of all before it.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                             const A &...args)
{
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_kv_write(const PagedCache &c, int cache_dtype, const void *k, const void *v,
                            int dtype, int B, int L, size_t k_stride, size_t v_stride,
                            const int32_t *page_table, int max_pages, const int32_t *start,
                            const int32_t *count, int *status, cudaStream_t s);
cudaError_t launch_kv_read(const PagedCache &c, int cache_dtype, const int32_t *page_table,
                           int max_pages, const int32_t *kv_len, int B, int L, void *k, void *v,
                           int dtype, int *status, cudaStream_t s);

// fp32 arithmetic throughout: the path of fp32 queries, row_block 4 or 8
constexpr int kPagedF32Tile = 64;
constexpr int paged_f32_per_sm(int row_block, bool e4m3) { return row_block == 8 ? 2 : e4m3 ? 4 : 3; }
cudaError_t launch_paged_f32(const PagedProblem &p, const PagedPart &part, int cache_dtype,
                             cudaStream_t s);

// bf16 queries, few rows: the keys as the M side of tcgen05 products.
// row_block * 128 / D is 8, 16, 24 or 32, a tile kPagedKeysTile rows of 128 values
// (with D = 64 two tokens each; boxes of min(page * D / 128, 128) rows)
constexpr int kPagedKeysTile = 128;
cudaError_t launch_paged_keys(const PagedProblem &p, const PagedPart &part, int cache_dtype,
                              const void *tm_k, const void *tm_v, cudaStream_t s);

// bf16 queries, D = 128, row_block 256: the rows as the M side (boxes of
// min(page, 64) tokens of an 8-bit cache, min(page, 128) of a 16-bit one)
constexpr int kPagedRowsTile = 128;
cudaError_t launch_paged_rows(const PagedProblem &p, const PagedPart &part, int cache_dtype,
                              const void *tm_k, const void *tm_v, cudaStream_t s);

// joins the partial results of both sources (n_parts of them) into out, lse
cudaError_t launch_paged_join(const PagedProblem &p, const PagedPart *parts, int n_parts, int dtype,
                              cudaStream_t s);

} // namespace ra
