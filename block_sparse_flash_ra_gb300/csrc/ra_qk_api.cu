// ra_qk_api.cu -- the C ABI of the norms and rotary positions of queries and
// keys (include/ra.h): argument checks and the workspace's layout.
#include "ra_args.h"
#include "ra_qk.h"

namespace ra {
namespace {

int check_qk(const ra_qk_params *p)
{
    if (!p) return refuse(RA_ERR_INVALID_ARG, "params is NULL");
    if (p->B <= 0 || p->L <= 0 || p->Hq < 0 || p->Hkv < 0 || p->Hq + (long long)p->Hkv == 0)
        return refuse(RA_ERR_INVALID_ARG, "sizes must be positive (B=%d L=%d Hq=%d Hkv=%d)", p->B, p->L, p->Hq, p->Hkv);
    if (p->D != 64 && p->D != 128) return refuse(RA_ERR_UNSUPPORTED, "D must be 64 or 128 (got %d)", p->D);
    if (p->dtype != RA_BF16 && p->dtype != RA_FP32)
        return refuse(RA_ERR_INVALID_ARG, "dtype must be RA_BF16 or RA_FP32");
    if (p->Hq > 65536 || p->Hkv > 65536) return refuse(RA_ERR_UNSUPPORTED, "at most 65536 heads");
    if ((double)p->B * p->L > 2147483647.0) return refuse(RA_ERR_UNSUPPORTED, "B * L must be below 2^31");
    const ra_rope &r = p->rope;
    if (r.rot < 0 || r.rot > p->D || r.rot % 16)
        return refuse(RA_ERR_UNSUPPORTED, "rot must be a multiple of 16 up to D (got %d of %d)", r.rot, p->D);
    if (r.rot && (!r.freq || !is_aligned(r.freq, 8)))
        return refuse(RA_ERR_INVALID_ARG, "a rotation needs its frequencies, 8-byte aligned");
    if (r.rot && !(r.amplitude > -1e30f && r.amplitude < 1e30f))
        return refuse(RA_ERR_INVALID_ARG, "amplitude must be finite");
    if (!(p->eps == 0.f || (p->eps >= 1e-30f && p->eps < 1e30f)))
        return refuse(RA_ERR_INVALID_ARG, "eps must be 0 (no norm), or at least 1e-30 and finite");
    if (p->eps == 0.f && (p->q_weight || p->k_weight))
        return refuse(RA_ERR_INVALID_ARG, "weights belong to a norm (eps > 0)");
    if (p->weight_dtype != RA_BF16 && p->weight_dtype != RA_FP32)
        return refuse(RA_ERR_INVALID_ARG, "weight_dtype must be RA_BF16 or RA_FP32");
    if (!is_aligned(p->pos, 4) || !is_aligned(p->start, 4) || !is_aligned(p->prefix_len, 4))
        return refuse(RA_ERR_INVALID_ARG, "pos, start and prefix_len must be 4-byte aligned");
    if (!is_aligned(p->q_weight, 16) || !is_aligned(p->k_weight, 16))
        return refuse(RA_ERR_INVALID_ARG, "weights must be 16-byte aligned");
    return RA_OK;
}

// A tensor of (tokens, heads, D) with its tokens `stride` elements apart.
struct Rows {
    const char *name;
    const void *p;
    size_t stride;
    int heads;
};

int check_rows(const ra_qk_params *p, const Rows &r)
{
    const size_t item = p->dtype == RA_BF16 ? 2 : 4, row = (size_t)r.heads * p->D;
    if (!r.p) return refuse(RA_ERR_INVALID_ARG, "%s is NULL", r.name);
    if (r.stride < row) return refuse(RA_ERR_INVALID_ARG, "%s: the stride must be at least heads * D (%zu)", r.name, row);
    if (!is_aligned(r.p, 16) || (r.stride * item) % 16)
        return refuse(RA_ERR_INVALID_ARG, "%s and its stride must be 16-byte aligned", r.name);
    return RA_OK;
}

// Whether an output may share memory with another tensor of the call: none of
// it, the other columns of the same rows, or -- an input that is read as the
// output is written -- exactly all of it.
bool may_share(const ra_qk_params *p, const Rows &out, const Rows &other, bool in_place)
{
    const size_t item = p->dtype == RA_BF16 ? 2 : 4, n = (size_t)p->B * p->L;
    const uintptr_t a = reinterpret_cast<uintptr_t>(out.p), b = reinterpret_cast<uintptr_t>(other.p);
    const size_t aw = (size_t)out.heads * p->D * item, bw = (size_t)other.heads * p->D * item;
    const size_t as = out.stride * item, bs = other.stride * item;
    if (!overlap(out.p, (n - 1) * as + aw, other.p, (n - 1) * bs + bw)) return true;
    if (as != bs) return false;
    if (a == b) return in_place && aw == bw;
    const size_t off = (a > b ? a - b : b - a) % as; // from the lower one's rows to the upper one's
    return a > b ? off >= bw && off + aw <= as : off >= aw && off + bw <= as;
}

int check_outputs(const ra_qk_params *p, const Rows *in, const int *own, int n_in, const Rows *out, int n_out)
{
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j) // own[j]: the output whose rows are made of this input's alone
            if (out[i].heads && in[j].heads && !may_share(p, out[i], in[j], own[j] == i))
                return refuse(RA_ERR_INVALID_ARG, "%s and %s overlap", out[i].name, in[j].name);
        for (int j = 0; j < i; ++j)
            if (out[i].heads && out[j].heads && !may_share(p, out[i], out[j], false))
                return refuse(RA_ERR_INVALID_ARG, "%s and %s overlap", out[i].name, out[j].name);
    }
    return RA_OK;
}

QkProblem problem_of(const ra_qk_params *p)
{
    QkProblem x{};
    x.B = p->B;
    x.L = p->L;
    x.Hq = p->Hq;
    x.Hkv = p->Hkv;
    x.D = p->D;
    x.rot = p->rope.rot;
    x.interleaved = p->rope.interleaved ? 1 : 0;
    x.amplitude = p->rope.amplitude;
    x.freq = p->rope.freq;
    x.pos = p->pos;
    x.start = p->start;
    x.prefix_len = p->prefix_len;
    x.eps = p->eps;
    x.weight_dtype = p->weight_dtype;
    x.q_weight = p->q_weight;
    x.k_weight = p->k_weight;
    return x;
}

QkRows rows_of(const Rows &r) { return {r.p, r.stride}; }

size_t bwd_bytes(const ra_qk_params *p) { return p->eps > 0.f ? (size_t)kQkBwdCtas * 2 * p->D * 4 : 0; }

} // namespace
} // namespace ra

using namespace ra;

extern "C" {

RA_API int ra_qk_fwd(const ra_qk_params *p, const void *q, size_t q_stride, const void *k, size_t k_stride, void *q_out,
                     size_t q_out_stride, void *k_out, size_t k_out_stride, ra_stream_t stream)
{
    int rc = check_qk(p);
    if (rc) return rc;
    const Rows in[2] = {{"q", q, q_stride, p->Hq}, {"k", k, k_stride, p->Hkv}};
    const Rows out[2] = {{"q_out", q_out, q_out_stride, p->Hq}, {"k_out", k_out, k_out_stride, p->Hkv}};
    const int own[2] = {0, 1};
    for (int i = 0; i < 2; ++i)
        if (in[i].heads && ((rc = check_rows(p, in[i])) || (rc = check_rows(p, out[i])))) return rc;
    if ((rc = check_outputs(p, in, own, 2, out, 2))) return rc;
    DeviceInfo d;
    if ((rc = device_info(&d))) return rc;
    const cudaError_t e = launch_qk_fwd(problem_of(p), p->dtype, p->eps > 0.f, rows_of(in[0]), rows_of(in[1]),
                                        rows_of(out[0]), rows_of(out[1]), reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_cuda_error(e, "qk forward launch");
    count_launches(1);
    return RA_OK;
}

RA_API size_t ra_qk_bwd_workspace_size(const ra_qk_params *p)
{
    return check_qk(p) == RA_OK ? bwd_bytes(p) : 0;
}

RA_API int ra_qk_bwd(const ra_qk_params *p, const void *q, size_t q_stride, const void *k, size_t k_stride,
                     const void *dq_out, size_t dq_out_stride, const void *dk_out, size_t dk_out_stride, void *dq,
                     size_t dq_stride, void *dk, size_t dk_stride, float *dq_weight, float *dk_weight, void *ws,
                     size_t ws_bytes, ra_stream_t stream)
{
    int rc = check_qk(p);
    if (rc) return rc;
    const bool norm = p->eps > 0.f;
    const Rows in[4] = {{"dq_out", dq_out, dq_out_stride, p->Hq}, {"dk_out", dk_out, dk_out_stride, p->Hkv},
                        {"q", q, q_stride, norm ? p->Hq : 0}, {"k", k, k_stride, norm ? p->Hkv : 0}};
    const Rows out[2] = {{"dq", dq, dq_stride, p->Hq}, {"dk", dk, dk_stride, p->Hkv}};
    const int own[4] = {0, 1, 0, 1};
    for (int i = 0; i < 4; ++i)
        if (in[i].heads && (rc = check_rows(p, in[i]))) return rc;
    for (int i = 0; i < 2; ++i)
        if (out[i].heads && (rc = check_rows(p, out[i]))) return rc;
    if ((rc = check_outputs(p, in, own, 4, out, 2))) return rc;
    if (!norm && (dq_weight || dk_weight)) return refuse(RA_ERR_INVALID_ARG, "weights belong to a norm (eps > 0)");
    if (norm) {
        if (dq_weight && dk_weight && overlap(dq_weight, (size_t)p->D * 4, dk_weight, (size_t)p->D * 4))
            return refuse(RA_ERR_INVALID_ARG, "dq_weight and dk_weight overlap"); // stored in no order
        if (!ws || ws_bytes < bwd_bytes(p))
            return refuse(RA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws ? ws_bytes : (size_t)0, bwd_bytes(p));
        if (!is_aligned(ws, 256)) return refuse(RA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
        if (!is_aligned(dq_weight, 4) || !is_aligned(dk_weight, 4))
            return refuse(RA_ERR_INVALID_ARG, "the weights' gradients must be 4-byte aligned");
    }
    DeviceInfo d;
    if ((rc = device_info(&d))) return rc;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    QkProblem x = problem_of(p);
    x.inverse = 1;
    const cudaError_t e =
        norm ? launch_qk_bwd(x, p->dtype, rows_of(in[2]), rows_of(in[3]), rows_of(in[0]), rows_of(in[1]), rows_of(out[0]),
                             rows_of(out[1]), dq_weight, dk_weight, static_cast<float *>(ws), d.index, s)
             : launch_qk_fwd(x, p->dtype, false, rows_of(in[0]), rows_of(in[1]), rows_of(out[0]), rows_of(out[1]), s);
    if (e != cudaSuccess) return set_cuda_error(e, "qk backward launch");
    count_launches(norm ? 2 : 1);
    return RA_OK;
}

RA_API int ra_qk_enter(const ra_qk_params *p, const ra_kv_cache *cache, const void *q, size_t q_stride, const void *k,
                       size_t k_stride, const void *v, size_t v_stride, void *q_out, size_t q_out_stride,
                       const int32_t *page_table, int max_pages, const int32_t *count, ra_stream_t stream)
{
    int rc = check_qk(p);
    if (rc || (rc = check_cache(cache))) return rc;
    if (p->Hkv != cache->Hkv || p->D != cache->D)
        return refuse(RA_ERR_INVALID_ARG, "the cache has %d kv heads of %d, the params %d of %d", cache->Hkv, cache->D,
                      p->Hkv, p->D);
    if (!page_table || max_pages <= 0 || !p->start)
        return refuse(RA_ERR_INVALID_ARG, "page_table, with max_pages > 0, and the params' start are needed");
    const Rows in[3] = {{"q", q, q_stride, p->Hq}, {"k", k, k_stride, p->Hkv}, {"v", v, v_stride, p->Hkv}};
    const Rows out{"q_out", q_out, q_out_stride, p->Hq};
    const int own[3] = {0, -1, -1};
    for (int i = 0; i < 3; ++i)
        if (in[i].heads && (rc = check_rows(p, in[i]))) return rc;
    if (p->Hq && (rc = check_rows(p, out))) return rc;
    if ((rc = check_outputs(p, in, own, 3, &out, 1))) return rc;
    DeviceInfo d;
    if ((rc = device_info(&d))) return rc;
    const QkEnter to{cache_of(cache), cache->dtype, page_table, max_pages, count, d.status};
    const cudaError_t e = launch_qk_enter(problem_of(p), p->dtype, p->eps > 0.f, rows_of(in[0]), rows_of(in[1]),
                                          rows_of(in[2]), rows_of(out), to, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_cuda_error(e, "qk enter launch");
    count_launches(1);
    return RA_OK;
}

} // extern "C"
