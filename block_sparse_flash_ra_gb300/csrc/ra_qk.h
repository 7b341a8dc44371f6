// ra_qk.h -- declarations shared by the entry points and kernels of the norms
// and rotary positions of queries and keys.
#pragma once

#include "ra_paged.h"

namespace ra {

struct QkProblem {
    int B, L, Hq, Hkv, D;
    // rotation: of the first `rot` values, pairs side by side or half of rot
    // apart; freq in turns per position, as fractions of 2^64
    int rot, interleaved, inverse;
    float amplitude;
    const uint64_t *freq;
    const int32_t *pos, *start, *prefix_len;
    // norm
    float eps;
    int weight_dtype;
    const void *q_weight, *k_weight; // NULL: ones
};

// One tensor of (tokens, heads, D) whose tokens are `stride` elements apart.
struct QkRows {
    const void *p;
    size_t stride;
};

// Where tokens enter a cache.
struct QkEnter {
    PagedCache c;
    int cache_dtype;
    const int32_t *table;
    int max_pages;
    const int32_t *count;
    int *status;
};

constexpr int kQkBwdCtas = 2 * 152; // of a backward with norms, at most
constexpr int kQkTokens = 8;        // of a CTA's step, at most

cudaError_t launch_qk_fwd(const QkProblem &p, int dtype, bool norm, QkRows q, QkRows k, QkRows q_out, QkRows k_out,
                          cudaStream_t s);
cudaError_t launch_qk_enter(const QkProblem &p, int dtype, bool norm, QkRows q, QkRows k, QkRows v, QkRows q_out,
                            const QkEnter &to, cudaStream_t s);
// with norms: part (kQkBwdCtas, 2, D) partial sums of the weights' gradients
cudaError_t launch_qk_bwd(const QkProblem &p, int dtype, QkRows q, QkRows k, QkRows dq_out, QkRows dk_out, QkRows dq,
                          QkRows dk, float *dq_weight, float *dk_weight, float *part, int device, cudaStream_t s);

} // namespace ra
