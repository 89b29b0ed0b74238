// Internal declarations of the paged-attention entry points (not public):
// launch arguments, and the device code shared by their kernels.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "kda_internal.cuh"
#include "kda_tc.cuh"

namespace kda {

// SMs of the current device (152 without one); asked once per device, since a call of
// a few microseconds notices the query.
int sm_count();

// Every kernel of these entry points is launched so that it may start while the kernel
// before it on the stream ends (programmatic dependent launch), and waits for that one,
// complete and its memory visible, ahead of its first access to global memory: in a chain
// of short calls the launches overlap (a decode of one request 15.4 -> 10.3 us a call, the
// append of 64 tokens 8.2 -> 4.9 us).  None of these signals early: blocks of the next kernel
// that wait beside it cost more than the signal saves (129 rotated tokens 6.9 instead of 4.8
// us).  Others do (the chunk scan), so nothing is held during the wait that a kernel may still
// have to allocate.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), cudaLaunchConfig_t cfg, cudaStream_t stream, A... args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}
__device__ __forceinline__ void wait_for_previous()
{
    tc::grid_dependency_wait();
}
inline cudaLaunchConfig_t launch_config(int64_t blocks, unsigned threads, size_t smem = 0)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    return cfg;
}

// ---------------------------------------------------------------- launches
struct PlanArgs {
    const int32_t* cached;
    const int32_t* cu;
    int32_t N;
    int32_t T;
    int32_t page;
    int32_t* table;
    int32_t max_pages;
    const int32_t* free_pages;
    int32_t num_free;
    const int32_t* free_start;
    int32_t* seq_lens;
    int32_t* positions;
    int64_t* slots;
    int32_t* free_end;
    int32_t* status;
};
cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t stream);

struct RopeArgs {
    const void* q;
    const void* k;
    const void* v;           // append only
    int32_t q_stride;        // elements between tokens
    int32_t k_stride;
    int32_t v_stride;
    bool x_bf16;
    const int32_t* positions;
    const float* inv_freq;
    int32_t rot;
    int32_t interleaved;
    float rope_scale;
    const float* q_weight;
    const float* k_weight;
    float eps;
    int32_t norm;
    int32_t T;
    int32_t Hq;
    int32_t Hk;
    int32_t D;
    void* q_out;             // forward: outputs; backward: q_grad, k_grad
    void* k_out;
    bool out_bf16;
    // append: k_out and v_out are the caches
    void* v_out;
    const int64_t* slots;
    int64_t num_slots;
    int32_t page;
    int32_t* status;
    // backward
    const void* dq;
    const void* dk;
    bool dy_bf16;
    float* q_wgrad;
    float* k_wgrad;
    float* partials;
};
cudaError_t launch_qk_rope(const RopeArgs& a, bool append, cudaStream_t stream);
cudaError_t launch_qk_rope_bwd(const RopeArgs& a, cudaStream_t stream);
int64_t qk_rope_bwd_workspace_bytes(int32_t D);

struct DecodeArgs {
    const void* q;
    const void* k;
    const void* v;
    bool bf16;
    const int32_t* table;
    const int32_t* seq_lens;
    int32_t N;
    const int32_t* live;     // requests from *live on have no row, whatever their lengths (nullptr: all have)
    int32_t Hq;
    int32_t Hk;
    int32_t D;
    int32_t num_pages;
    int32_t page_shift;
    int32_t max_pages;
    float scale;
    void* out;
    bool out_bf16;
    float* lse;
    void* workspace;
    int32_t* status;
};
int64_t paged_decode_workspace_bytes(int32_t N, int32_t Hq, int32_t Hk, int32_t D);
cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t stream);

// ---------------------------------------------------------------- pairs of FP32
__device__ __forceinline__ uint64_t as_u64(float2 x)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x.x), "f"(x.y));
    return r;
}
__device__ __forceinline__ float2 as_f2(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
    return as_f2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

}  // namespace kda
