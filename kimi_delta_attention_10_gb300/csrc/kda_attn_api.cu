// Host side of the entry points of attention for several tokens declared in
// include/kda.h: argument validation and dispatch.  Nothing is launched unless every
// host-visible check passes.
#include <cuda_runtime.h>
#include <initializer_list>
#include <stdint.h>

#include "kda.h"
#include "kda_attn.cuh"

namespace {

bool valid_dtype(int32_t d) { return d == KDA_F32 || d == KDA_BF16; }
kda_status result(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }
bool all_aligned(std::initializer_list<const void*> ptrs, uintptr_t to = 16)
{
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return false;
    return true;
}
// Arrays of integers are read one at a time, so that a row of a table or a slice will do.
bool ints_aligned(std::initializer_list<const void*> ptrs) { return all_aligned(ptrs, 4); }
// Every output given is none of the inputs and no other output (by base pointer).
bool apart(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins)
{
    for (const void* const* o = outs.begin(); o != outs.end(); ++o) {
        if (!*o) continue;
        for (const void* p : ins)
            if (p == *o) return false;
        for (const void* const* x = o + 1; x != outs.end(); ++x)
            if (*x == *o) return false;
    }
    return true;
}
int64_t aligned(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Sizes that all of these entry points have.
kda_status check_sizes(int32_t N, int64_t T, int32_t Hq, int32_t Hk, int32_t D)
{
    if (N < 0 || T < 0 || Hq < 1 || Hk < 1 || D < 1) return KDA_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || Hq % Hk != 0) return KDA_ERR_UNSUPPORTED;
    // N: every CTA looks at all offsets; T by itself first, since T + N could wrap
    if (N > (1 << 16) || T > INT32_MAX || T + N > INT32_MAX / Hq || Hq > INT32_MAX / D) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
kda_status check_cache(int32_t Hk, int32_t num_pages, int32_t page_size, int32_t max_pages)
{
    if (num_pages < 0 || page_size < 1 || max_pages < 1) return KDA_ERR_INVALID_ARG;
    if ((page_size & (page_size - 1)) != 0 || page_size < 8 || page_size > 1024) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)num_pages * Hk > INT32_MAX / page_size) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
// The strides of packed rows: at least the heads, whole 16 bytes.
kda_status check_stride(int64_t stride, int32_t H, int32_t D, int32_t dtype)
{
    if (stride < (int64_t)H * D) return KDA_ERR_INVALID_ARG;
    if (stride > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    return stride * (dtype == KDA_BF16 ? 2 : 4) % 16 ? KDA_ERR_ALIGNMENT : KDA_OK;
}

kda::AttnArgs common(int32_t dtype, int32_t N, int64_t T, int32_t Hq, int32_t Hk, int32_t D, float scale)
{
    kda::AttnArgs a = {};
    a.bf16 = dtype == KDA_BF16;
    a.N = N; a.T = (int32_t)T; a.Hq = Hq; a.Hk = Hk; a.D = D; a.scale = scale;
    a.causal = true;
    a.splits = a.pieces = 1;
    a.fault = kda::test_fault();
    return a;
}

// Bytes for the pieces of a call (`more` of them beside the forward's), whatever its
// lengths and type; 16 where it needs none.
int64_t pieces_bytes(int32_t N, int64_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t more)
{
    kda::AttnArgs a = common(KDA_F32, N, T, Hq, Hk, D, 0.f);
    int64_t most = 16;
    for (bool bf16 : {false, true}) {
        a.pieces = kda::attn_splits(bf16, N, a.T, Hq, Hk, D, INT64_MAX) + more;
        const int64_t b = a.pieces > 1 ? kda::attn_pieces_o(a, a.pieces) : 0;
        if (b > most) most = b;
    }
    return aligned(most);
}

// The forward, in as many pieces as fill the GPU, and their join.
kda_status attend(kda::AttnArgs& a, int64_t kv_most, cudaStream_t stream)
{
    a.splits = a.pieces = kda::attn_splits(a.bf16, a.N, a.T, a.Hq, a.Hk, a.D, kv_most);
    cudaError_t e = kda::launch_attention(a, stream);
    if (e == cudaSuccess && a.pieces > 1) e = kda::launch_attn_join(a, stream);
    return result(e);
}

}  // namespace

extern "C" {

kda_status kda_attention_workspace_size(int32_t N, int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                                        int64_t* bytes_host)
{
    if (!bytes_host) return KDA_ERR_INVALID_ARG;
    const kda_status st = check_sizes(N, T, Hq, Hk, D);
    if (st == KDA_OK) *bytes_host = pieces_bytes(N, T, Hq, Hk, D, 0);
    return st;
}

kda_status kda_attention_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, int32_t dtype,
                             const int32_t* cu_seqlens, int32_t N, int64_t T, int32_t Hq,
                             int32_t Hk, int32_t D, float scale, void* out, float* lse,
                             void* workspace, int64_t workspace_bytes, int32_t* status_dev,
                             kda_stream_t stream)
{
    kda_status st = check_sizes(N, T, Hq, Hk, D);
    if (st != KDA_OK) return st;
    if (!valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    if ((st = check_stride(q_stride, Hq, D, dtype)) != KDA_OK) return st;
    if ((st = check_stride(k_stride, Hk, D, dtype)) != KDA_OK) return st;
    if ((st = check_stride(v_stride, Hk, D, dtype)) != KDA_OK) return st;
    if (T == 0 || N == 0) return KDA_OK;
    if (!q || !k || !v || !cu_seqlens || !out || !workspace) return KDA_ERR_INVALID_ARG;
    if (!all_aligned({q, k, v, out, lse, workspace}) || !ints_aligned({cu_seqlens, status_dev}))
        return KDA_ERR_ALIGNMENT;
    if (!apart({out, lse, workspace}, {q, k, v, cu_seqlens})) return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < pieces_bytes(N, T, Hq, Hk, D, 0)) return KDA_ERR_INVALID_ARG;
    kda::AttnArgs a = common(dtype, N, T, Hq, Hk, D, scale);
    a.q = q; a.k = k; a.v = v;
    a.q_stride = (int32_t)q_stride; a.k_stride = (int32_t)k_stride; a.v_stride = (int32_t)v_stride;
    a.cu = cu_seqlens; a.out = out; a.lse = lse; a.workspace = workspace; a.status = status_dev;
    return attend(a, T, reinterpret_cast<cudaStream_t>(stream));
}

kda_status kda_attention_bwd_workspace_size(int32_t N, int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                                            int64_t* bytes_host)
{
    if (!bytes_host) return KDA_ERR_INVALID_ARG;
    const kda_status st = check_sizes(N, T, Hq, Hk, D);
    if (st == KDA_OK) *bytes_host = kda::attention_bwd_workspace_bytes(N, (int32_t)T, Hq, Hk, D);
    return st;
}

kda_status kda_attention_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, int32_t dtype, const void* out,
                             const float* lse, const void* dout, const int32_t* cu_seqlens,
                             int32_t N, int64_t T, int32_t Hq, int32_t Hk, int32_t D, float scale,
                             void* q_grad, void* k_grad, void* v_grad, void* workspace,
                             int64_t workspace_bytes, int32_t* status_dev, kda_stream_t stream)
{
    kda_status st = check_sizes(N, T, Hq, Hk, D);
    if (st != KDA_OK) return st;
    if (!valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    if ((st = check_stride(q_stride, Hq, D, dtype)) != KDA_OK) return st;
    if ((st = check_stride(k_stride, Hk, D, dtype)) != KDA_OK) return st;
    if ((st = check_stride(v_stride, Hk, D, dtype)) != KDA_OK) return st;
    if (T == 0 || N == 0) return KDA_OK;
    if (!q || !k || !v || !out || !lse || !dout || !cu_seqlens || !q_grad || !k_grad || !v_grad || !workspace)
        return KDA_ERR_INVALID_ARG;
    if (!all_aligned({q, k, v, out, lse, dout, q_grad, k_grad, v_grad, workspace}) ||
        !ints_aligned({cu_seqlens, status_dev}))
        return KDA_ERR_ALIGNMENT;
    if (!apart({q_grad, k_grad, v_grad, workspace}, {q, k, v, out, lse, dout, cu_seqlens}))
        return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < kda::attention_bwd_workspace_bytes(N, (int32_t)T, Hq, Hk, D)) return KDA_ERR_INVALID_ARG;
    kda::AttnArgs a = common(dtype, N, T, Hq, Hk, D, scale);
    a.q = q; a.k = k; a.v = v;
    a.q_stride = (int32_t)q_stride; a.k_stride = (int32_t)k_stride; a.v_stride = (int32_t)v_stride;
    a.cu = cu_seqlens; a.out = const_cast<void*>(out); a.lse_in = lse; a.dout = dout;
    a.dq = q_grad; a.dk = k_grad; a.dv = v_grad; a.workspace = workspace; a.status = status_dev;
    return result(kda::launch_attention_bwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_paged_prompt_workspace_size(int32_t N, int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                                           int64_t* bytes_host)
{
    return kda_attention_workspace_size(N, T, Hq, Hk, D, bytes_host);
}

kda_status kda_paged_prompt(const void* q, int64_t q_stride, const void* k_cache,
                            const void* v_cache, int32_t dtype, const int32_t* block_table,
                            const int32_t* seq_lens, const int32_t* cu_seqlens, int32_t N,
                            int64_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t num_pages,
                            int32_t page_size, int32_t max_pages, float scale, void* out,
                            float* lse, void* workspace, int64_t workspace_bytes,
                            int32_t* status_dev, kda_stream_t stream)
{
    kda_status st = check_sizes(N, T, Hq, Hk, D);
    if (st != KDA_OK) return st;
    if (!valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    if ((st = check_stride(q_stride, Hq, D, dtype)) != KDA_OK) return st;
    if ((st = check_cache(Hk, num_pages, page_size, max_pages)) != KDA_OK) return st;
    if (T == 0 || N == 0) return KDA_OK;
    if (!q || !block_table || !seq_lens || !cu_seqlens || !out || !workspace) return KDA_ERR_INVALID_ARG;
    if (num_pages > 0 && (!k_cache || !v_cache)) return KDA_ERR_INVALID_ARG;
    if (!all_aligned({q, k_cache, v_cache, out, lse, workspace}) ||
        !ints_aligned({block_table, seq_lens, cu_seqlens, status_dev}))
        return KDA_ERR_ALIGNMENT;
    if (!apart({out, lse, workspace}, {q, k_cache, v_cache, block_table, seq_lens, cu_seqlens}))
        return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < pieces_bytes(N, T, Hq, Hk, D, 0)) return KDA_ERR_INVALID_ARG;
    kda::AttnArgs a = common(dtype, N, T, Hq, Hk, D, scale);
    a.q = q; a.q_stride = (int32_t)q_stride; a.k = k_cache; a.v = v_cache; a.cu = cu_seqlens;
    a.table = block_table; a.kv_lens = seq_lens; a.num_pages = num_pages; a.max_pages = max_pages;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.out = out; a.lse = lse; a.workspace = workspace; a.status = status_dev;
    return attend(a, (int64_t)max_pages * page_size, reinterpret_cast<cudaStream_t>(stream));
}

kda_status kda_paged_decode_shared_workspace_size(int32_t N, int32_t groups, int32_t Hq, int32_t Hk,
                                                  int32_t D, int64_t* bytes_host)
{
    if (!bytes_host || groups < 0) return KDA_ERR_INVALID_ARG;
    kda_status st = check_sizes(groups, N, Hq, Hk, D);
    if (st != KDA_OK) return st;
    *bytes_host = pieces_bytes(groups, N, Hq, Hk, D, 1) + kda::paged_decode_workspace_bytes(N, Hq, Hk, D);
    return KDA_OK;
}

kda_status kda_paged_decode_shared(const void* q, const void* k_cache, const void* v_cache,
                                   int32_t dtype, const int32_t* prefix_table,
                                   const int32_t* prefix_lens, const int32_t* cu_groups,
                                   int32_t groups, int32_t max_prefix_pages,
                                   const int32_t* block_table, const int32_t* seq_lens, int32_t N,
                                   int32_t Hq, int32_t Hk, int32_t D, int32_t num_pages,
                                   int32_t page_size, int32_t max_pages, float scale, void* out,
                                   float* lse, void* workspace, int64_t workspace_bytes,
                                   int32_t* status_dev, kda_stream_t stream)
{
    if (groups < 0) return KDA_ERR_INVALID_ARG;
    kda_status st = check_sizes(groups, N, Hq, Hk, D);
    if (st != KDA_OK) return st;
    if (!valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    if ((st = check_cache(Hk, num_pages, page_size, max_pages)) != KDA_OK) return st;
    if (max_prefix_pages < 1) return KDA_ERR_INVALID_ARG;
    if (N == 0 || groups == 0) return KDA_OK;
    if (!q || !prefix_table || !prefix_lens || !cu_groups || !block_table || !seq_lens || !out || !workspace)
        return KDA_ERR_INVALID_ARG;
    if (num_pages > 0 && (!k_cache || !v_cache)) return KDA_ERR_INVALID_ARG;
    if (!all_aligned({q, k_cache, v_cache, out, lse, workspace}) ||
        !ints_aligned({prefix_table, prefix_lens, cu_groups, block_table, seq_lens, status_dev}))
        return KDA_ERR_ALIGNMENT;
    if (!apart({out, lse, workspace},
               {q, k_cache, v_cache, prefix_table, prefix_lens, cu_groups, block_table, seq_lens}))
        return KDA_ERR_INVALID_ARG;
    const int64_t pieces = pieces_bytes(groups, N, Hq, Hk, D, 1);
    if (workspace_bytes < pieces + kda::paged_decode_workspace_bytes(N, Hq, Hk, D)) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    // the prefix: its group's requests are the tokens of one sequence, all of which see all of it
    kda::AttnArgs a = common(dtype, groups, N, Hq, Hk, D, scale);
    a.causal = false;
    a.q = q; a.q_stride = Hq * D; a.k = k_cache; a.v = v_cache; a.cu = cu_groups;
    a.table = prefix_table; a.kv_lens = prefix_lens; a.num_pages = num_pages; a.max_pages = max_prefix_pages;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.out = out; a.lse = lse; a.workspace = workspace; a.status = status_dev;
    a.splits = kda::attn_splits(a.bf16, a.N, a.T, Hq, Hk, D, (int64_t)max_prefix_pages * page_size);
    a.pieces = a.splits + 1;
    cudaError_t e = kda::launch_attention(a, s);
    if (e != cudaSuccess) return result(e);

    // the last piece: every request's own tokens
    char* ws = static_cast<char*>(workspace);
    kda::DecodeArgs d = {};
    d.q = q; d.k = k_cache; d.v = v_cache; d.bf16 = a.bf16; d.table = block_table; d.seq_lens = seq_lens;
    d.N = N; d.live = cu_groups + groups;
    d.Hq = Hq; d.Hk = Hk; d.D = D; d.num_pages = num_pages; d.page_shift = a.page_shift;
    d.max_pages = max_pages; d.scale = scale;
    d.out = ws + kda::attn_pieces_o(a, a.splits);
    d.lse = reinterpret_cast<float*>(ws + kda::attn_pieces_lse(a, a.splits));
    d.workspace = ws + pieces; d.status = status_dev;
    e = kda::launch_paged_decode(d, s);
    if (e == cudaSuccess) e = kda::launch_attn_join(a, s);
    return result(e);
}

}  // extern "C"
