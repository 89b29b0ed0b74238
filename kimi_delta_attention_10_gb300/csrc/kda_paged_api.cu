// Host side of the paged-attention entry points declared in include/kda.h:
// argument validation and dispatch.  Nothing is launched unless every
// host-visible check passes.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "kda_paged.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool valid_dtype(int32_t d) { return d == KDA_F32 || d == KDA_BF16; }
int64_t dtype_size(int32_t d) { return d == KDA_BF16 ? 2 : 4; }
bool valid_head(int32_t D) { return D == 64 || D == 128; }

template <int N> bool all_aligned(const void* const (&ptrs)[N])
{
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return false;
    return true;
}

kda_status result(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// What the three norm-and-rotation entry points have in common; KDA_OK fills `r`.
kda_status check_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      int32_t x_dtype, const int32_t* positions, const float* inv_freq,
                      int32_t rot_dim, int32_t interleaved, float rope_scale,
                      const float* q_weight, const float* k_weight, float eps, int32_t qk_norm,
                      int64_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t out_dtype,
                      kda::RopeArgs* r)
{
    if (T < 0 || Hq < 1 || Hk < 1 || D < 1 || rot_dim < 0) return KDA_ERR_INVALID_ARG;
    if (!valid_dtype(x_dtype) || !valid_dtype(out_dtype)) return KDA_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return KDA_ERR_INVALID_ARG;
    if (qk_norm != 0 && qk_norm != 1) return KDA_ERR_INVALID_ARG;
    if (qk_norm && !(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (T > INT32_MAX || !valid_head(D)) return KDA_ERR_UNSUPPORTED;
    if (rot_dim % 16 != 0 || rot_dim > D) return KDA_ERR_UNSUPPORTED;
    if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hk * D) return KDA_ERR_INVALID_ARG;
    if (q_stride > INT32_MAX || k_stride > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const int64_t es = dtype_size(x_dtype);
    if (q_stride * es % 16 != 0 || k_stride * es % 16 != 0) return KDA_ERR_ALIGNMENT;
    if (T > 0 && (!q || !k || !positions)) return KDA_ERR_INVALID_ARG;
    if (T > 0 && rot_dim > 0 && !inv_freq) return KDA_ERR_INVALID_ARG;
    if (!all_aligned({q, k, static_cast<const void*>(positions), static_cast<const void*>(inv_freq),
                      static_cast<const void*>(q_weight), static_cast<const void*>(k_weight)}))
        return KDA_ERR_ALIGNMENT;
    *r = {};
    r->q = q; r->k = k; r->q_stride = (int32_t)q_stride;
    r->k_stride = (int32_t)k_stride;
    r->x_bf16 = x_dtype == KDA_BF16; r->positions = positions; r->inv_freq = inv_freq;
    r->rot = rot_dim; r->interleaved = interleaved; r->rope_scale = rope_scale;
    r->q_weight = q_weight; r->k_weight = k_weight; r->eps = eps; r->norm = qk_norm;
    r->T = (int32_t)T; r->Hq = Hq; r->Hk = Hk; r->D = D; r->out_bf16 = out_dtype == KDA_BF16;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_page_plan(const int32_t* cached_lens, const int32_t* cu_seqlens, int32_t N,
                         int64_t T, int32_t page_size, int32_t* block_table, int32_t max_pages,
                         const int32_t* free_pages, int32_t num_free, const int32_t* free_start,
                         int32_t* seq_lens, int32_t* positions, int64_t* slots,
                         int32_t* free_end, int32_t* status_dev, kda_stream_t stream)
{
    if (N < 0 || T < 0 || page_size < 1 || max_pages < 1 || num_free < 0)
        return KDA_ERR_INVALID_ARG;
    if (T > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (N == 0 && T > 0) return KDA_ERR_INVALID_ARG;
    if (!free_end) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (!cached_lens || !cu_seqlens || !block_table || !seq_lens))
        return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!positions || !slots)) return KDA_ERR_INVALID_ARG;
    if (num_free > 0 && !free_pages) return KDA_ERR_INVALID_ARG;
    // single integers are read and written: their natural alignment is enough
    for (const void* p : {static_cast<const void*>(cached_lens), static_cast<const void*>(cu_seqlens),
                          static_cast<const void*>(block_table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_start), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(positions), static_cast<const void*>(free_end),
                          static_cast<const void*>(status_dev)})
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return KDA_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(slots) % 8 != 0)
        return KDA_ERR_ALIGNMENT;
    // no output may be an input or another output (checked on the base pointers)
    const void* outs[] = {block_table, seq_lens, positions, slots, free_end};
    const void* ins[] = {cached_lens, cu_seqlens, free_pages, free_start};
    for (int i = 0; i < 5; ++i) {
        if (!outs[i]) continue;
        for (const void* p : ins)
            if (p == outs[i]) return KDA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 5; ++j)
            if (outs[j] == outs[i]) return KDA_ERR_INVALID_ARG;
    }
    kda::PlanArgs a = {};
    a.cached = cached_lens; a.cu = cu_seqlens; a.N = N; a.T = (int32_t)T; a.page = page_size;
    a.table = block_table; a.max_pages = max_pages; a.free_pages = free_pages;
    a.num_free = num_free; a.free_start = free_start; a.seq_lens = seq_lens;
    a.positions = positions; a.slots = slots; a.free_end = free_end; a.status = status_dev;
    return result(kda::launch_page_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_rope_inv_freq(int32_t rot_dim, double theta, int32_t scaling, double factor,
                             double original_len, double beta_fast, double beta_slow,
                             float* inv_freq_host, float* rope_scale_host)
{
    if (rot_dim < 2 || rot_dim % 2 != 0 || !(theta > 1.0)) return KDA_ERR_INVALID_ARG;
    if (!inv_freq_host || !rope_scale_host) return KDA_ERR_INVALID_ARG;
    if (scaling < KDA_ROPE_PLAIN || scaling > KDA_ROPE_YARN) return KDA_ERR_INVALID_ARG;
    if (scaling != KDA_ROPE_PLAIN && !(factor >= 1.0)) return KDA_ERR_INVALID_ARG;
    if (scaling == KDA_ROPE_NTK && rot_dim < 4) return KDA_ERR_INVALID_ARG;
    if (scaling == KDA_ROPE_YARN &&
        !(original_len > 0.0 && beta_slow > 0.0 && beta_fast > beta_slow))
        return KDA_ERR_INVALID_ARG;
    const int pairs = rot_dim / 2;
    const double two_pi = 6.283185307179586476925;
    double base = theta;
    if (scaling == KDA_ROPE_NTK) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    // the (fractional) pair that turns `beta` times in original_len tokens
    auto pair_of = [&](double beta) {
        return pairs * log(original_len / (two_pi * beta)) / log(theta);
    };
    double lo = 0.0, hi = 0.0;
    if (scaling == KDA_ROPE_YARN) {
        lo = fmax(floor(pair_of(beta_fast)), 0.0);
        hi = fmin(ceil(pair_of(beta_slow)), rot_dim - 1.0);
    }
    for (int i = 0; i < pairs; ++i) {
        double f = pow(base, -(double)i / pairs);
        if (scaling == KDA_ROPE_LINEAR) f /= factor;
        if (scaling == KDA_ROPE_YARN) {
            // 1: interpolated, 0: kept
            const double slow = i >= hi ? 1.0 : i <= lo ? 0.0 : (i - lo) / (hi - lo);
            f = f * (1.0 - slow) + f / factor * slow;
        }
        inv_freq_host[i] = (float)f;
    }
    *rope_scale_host = scaling == KDA_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    return KDA_OK;
}

kda_status kda_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            int32_t x_dtype, const int32_t* positions, const float* inv_freq,
                            int32_t rot_dim, int32_t interleaved, float rope_scale,
                            const float* q_weight, const float* k_weight, float eps,
                            int32_t qk_norm, int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                            void* q_out, void* k_out, int32_t out_dtype, kda_stream_t stream)
{
    kda::RopeArgs a;
    kda_status st = check_rope(q, q_stride, k, k_stride, x_dtype, positions, inv_freq, rot_dim,
                               interleaved, rope_scale, q_weight, k_weight, eps, qk_norm, T, Hq,
                               Hk, D, out_dtype, &a);
    if (st != KDA_OK) return st;
    if (T > 0 && (!q_out || !k_out)) return KDA_ERR_INVALID_ARG;
    if (!all_aligned({static_cast<const void*>(q_out), static_cast<const void*>(k_out)}))
        return KDA_ERR_ALIGNMENT;
    if (T == 0) return KDA_OK;
    if (q_out == k_out || q_out == k || k_out == q) return KDA_ERR_INVALID_ARG;
    const bool same = x_dtype == out_dtype;
    if (q_out == q && (!same || q_stride != (int64_t)Hq * D)) return KDA_ERR_INVALID_ARG;
    if (k_out == k && (!same || k_stride != (int64_t)Hk * D)) return KDA_ERR_INVALID_ARG;
    a.q_out = q_out; a.k_out = k_out;
    return result(kda::launch_qk_rope(a, false, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k,
                                   int64_t k_stride, const void* v, int64_t v_stride,
                                   int32_t x_dtype, const int32_t* positions,
                                   const int64_t* slots, const float* inv_freq, int32_t rot_dim,
                                   int32_t interleaved, float rope_scale, const float* q_weight,
                                   const float* k_weight, float eps, int32_t qk_norm, int64_t T,
                                   int32_t Hq, int32_t Hk, int32_t D, void* q_out, void* k_cache,
                                   void* v_cache, int32_t cache_dtype, int32_t num_pages,
                                   int32_t page_size, int32_t* status_dev, kda_stream_t stream)
{
    kda::RopeArgs a;
    kda_status st = check_rope(q, q_stride, k, k_stride, x_dtype, positions, inv_freq, rot_dim,
                               interleaved, rope_scale, q_weight, k_weight, eps, qk_norm, T, Hq,
                               Hk, D, cache_dtype, &a);
    if (st != KDA_OK) return st;
    if (num_pages < 0 || page_size < 1) return KDA_ERR_INVALID_ARG;
    if (v_stride < (int64_t)Hk * D) return KDA_ERR_INVALID_ARG;
    if (v_stride > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (v_stride * dtype_size(x_dtype) % 16 != 0) return KDA_ERR_ALIGNMENT;
    if (T > 0 && (!v || !slots || !q_out)) return KDA_ERR_INVALID_ARG;
    if (T > 0 && num_pages > 0 && (!k_cache || !v_cache)) return KDA_ERR_INVALID_ARG;
    if (!all_aligned({v, static_cast<const void*>(slots), static_cast<const void*>(q_out),
                      static_cast<const void*>(k_cache), static_cast<const void*>(v_cache),
                      static_cast<const void*>(status_dev)}))
        return KDA_ERR_ALIGNMENT;
    if (T == 0) return KDA_OK;
    if (q_out == q && (x_dtype != cache_dtype || q_stride != (int64_t)Hq * D))
        return KDA_ERR_INVALID_ARG;
    const void* outs[] = {q_out, k_cache, v_cache};
    const void* ins[] = {k, v, positions, slots};
    for (int i = 0; i < 3; ++i) {
        if (!outs[i]) continue;
        for (const void* p : ins)
            if (p == outs[i]) return KDA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (outs[j] == outs[i]) return KDA_ERR_INVALID_ARG;
        if (i > 0 && outs[i] == q) return KDA_ERR_INVALID_ARG;
    }
    a.v = v; a.v_stride = (int32_t)v_stride; a.slots = slots; a.q_out = q_out; a.k_out = k_cache;
    a.v_out = v_cache; a.page = page_size; a.num_slots = (int64_t)num_pages * page_size;
    a.status = status_dev;
    return result(kda::launch_qk_rope(a, true, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_qk_norm_rope_bwd_workspace_size(int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                                               int64_t* bytes_host)
{
    if (!bytes_host || T < 0 || Hq < 1 || Hk < 1 || D < 1) return KDA_ERR_INVALID_ARG;
    if (T > INT32_MAX || !valid_head(D)) return KDA_ERR_UNSUPPORTED;
    *bytes_host = kda::qk_rope_bwd_workspace_bytes(D);
    return KDA_OK;
}

kda_status kda_qk_norm_rope_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                int32_t x_dtype, const void* dq_out, const void* dk_out,
                                int32_t dy_dtype, const int32_t* positions,
                                const float* inv_freq, int32_t rot_dim, int32_t interleaved,
                                float rope_scale, const float* q_weight, const float* k_weight,
                                float eps, int32_t qk_norm, int64_t T, int32_t Hq, int32_t Hk,
                                int32_t D, void* q_grad, void* k_grad, int32_t grad_dtype,
                                float* q_weight_grad, float* k_weight_grad, void* workspace,
                                int64_t workspace_bytes, kda_stream_t stream)
{
    kda::RopeArgs a;
    kda_status st = check_rope(q, q_stride, k, k_stride, x_dtype, positions, inv_freq, rot_dim,
                               interleaved, rope_scale, q_weight, k_weight, eps, qk_norm, T, Hq,
                               Hk, D, grad_dtype, &a);
    if (st != KDA_OK) return st;
    if (!valid_dtype(dy_dtype)) return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!dq_out || !dk_out || !q_grad || !k_grad)) return KDA_ERR_INVALID_ARG;
    const bool sums = qk_norm && (q_weight_grad || k_weight_grad);
    if (sums && (!workspace || workspace_bytes < kda::qk_rope_bwd_workspace_bytes(D)))
        return KDA_ERR_INVALID_ARG;
    if (!all_aligned({dq_out, dk_out, static_cast<const void*>(q_grad),
                      static_cast<const void*>(k_grad), static_cast<const void*>(q_weight_grad),
                      static_cast<const void*>(k_weight_grad),
                      static_cast<const void*>(workspace)}))
        return KDA_ERR_ALIGNMENT;
    // no output may be an input or another output (checked on the base pointers),
    // except a gradient written over the one it is computed from
    const void* outs[] = {q_grad, k_grad, q_weight_grad, k_weight_grad, workspace};
    const void* ins[] = {q, k, dq_out, dk_out, positions, inv_freq, q_weight, k_weight};
    for (int i = 0; i < 5; ++i) {
        if (!outs[i]) continue;
        for (const void* p : ins) {
            if (p != outs[i]) continue;
            const bool over = (i == 0 && p == dq_out && p != dk_out) ||
                              (i == 1 && p == dk_out && p != dq_out);
            if (!over || dy_dtype != grad_dtype) return KDA_ERR_INVALID_ARG;
        }
        for (int j = i + 1; j < 5; ++j)
            if (outs[j] == outs[i]) return KDA_ERR_INVALID_ARG;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        // no tokens: the weights' gradients are zero
        cudaError_t e = cudaSuccess;
        for (float* w : {q_weight_grad, k_weight_grad})
            if (qk_norm && w && e == cudaSuccess) e = cudaMemsetAsync(w, 0, (size_t)D * 4, s);
        return result(e);
    }
    a.dq = dq_out; a.dk = dk_out; a.dy_bf16 = dy_dtype == KDA_BF16;
    a.q_out = q_grad; a.k_out = k_grad; a.q_wgrad = q_weight_grad; a.k_wgrad = k_weight_grad;
    a.partials = static_cast<float*>(workspace);
    return result(kda::launch_qk_rope_bwd(a, s));
}

namespace {

kda_status check_decode_sizes(int32_t N, int32_t Hq, int32_t Hk, int32_t D)
{
    if (N < 0 || Hq < 1 || Hk < 1 || D < 1) return KDA_ERR_INVALID_ARG;
    if (!valid_head(D) || Hq % Hk != 0) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)N * Hq > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

kda_status kda_paged_decode_workspace_size(int32_t N, int32_t Hq, int32_t Hk, int32_t D,
                                           int64_t* bytes_host)
{
    if (!bytes_host) return KDA_ERR_INVALID_ARG;
    kda_status st = check_decode_sizes(N, Hq, Hk, D);
    if (st == KDA_OK) *bytes_host = kda::paged_decode_workspace_bytes(N, Hq, Hk, D);
    return st;
}

kda_status kda_paged_decode(const void* q, const void* k_cache, const void* v_cache,
                            int32_t dtype, const int32_t* block_table, const int32_t* seq_lens,
                            int32_t N, int32_t Hq, int32_t Hk, int32_t D, int32_t num_pages,
                            int32_t page_size, int32_t max_pages, float scale, void* out,
                            int32_t out_dtype, float* lse, void* workspace,
                            int64_t workspace_bytes, int32_t* status_dev, kda_stream_t stream)
{
    kda_status st = check_decode_sizes(N, Hq, Hk, D);
    if (st != KDA_OK) return st;
    if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return KDA_ERR_INVALID_ARG;
    if (num_pages < 0 || page_size < 1 || max_pages < 1) return KDA_ERR_INVALID_ARG;
    if ((page_size & (page_size - 1)) != 0 || page_size < 8 || page_size > 1024)
        return KDA_ERR_UNSUPPORTED;
    if ((int64_t)num_pages * Hk > INT32_MAX / page_size) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    if (!q || !block_table || !seq_lens || !out || !workspace) return KDA_ERR_INVALID_ARG;
    if (num_pages > 0 && (!k_cache || !v_cache)) return KDA_ERR_INVALID_ARG;
    if (!all_aligned({q, k_cache, v_cache, static_cast<const void*>(block_table),
                      static_cast<const void*>(seq_lens), static_cast<const void*>(out),
                      static_cast<const void*>(lse), static_cast<const void*>(workspace),
                      static_cast<const void*>(status_dev)}))
        return KDA_ERR_ALIGNMENT;
    if (workspace_bytes < kda::paged_decode_workspace_bytes(N, Hq, Hk, D))
        return KDA_ERR_INVALID_ARG;
    const void* outs[] = {out, lse, workspace};
    const void* ins[] = {q, k_cache, v_cache, block_table, seq_lens};
    for (int i = 0; i < 3; ++i) {
        if (!outs[i]) continue;
        for (const void* p : ins)
            if (p == outs[i]) return KDA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (outs[j] == outs[i]) return KDA_ERR_INVALID_ARG;
    }
    kda::DecodeArgs a = {};
    a.q = q; a.k = k_cache; a.v = v_cache; a.bf16 = dtype == KDA_BF16; a.table = block_table;
    a.seq_lens = seq_lens; a.N = N; a.Hq = Hq; a.Hk = Hk; a.D = D; a.num_pages = num_pages;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.max_pages = max_pages; a.scale = scale; a.out = out; a.out_bf16 = out_dtype == KDA_BF16;
    a.lse = lse; a.workspace = workspace; a.status = status_dev;
    return result(kda::launch_paged_decode(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
