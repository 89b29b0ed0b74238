// What the tensor-core kernels of attention for several tokens share: products with an
// operand in tensor memory, wide tensor-memory loads and stores, tiles of rows and keys by TMA.
#pragma once

#include <cuda.h>
#include <math_constants.h>
#include <stdint.h>
#include <string.h>

#include "kda_attn.cuh"
#include "kda_paged_tma.cuh"

namespace kda {

constexpr float kAttnLog2e = 1.4426950408889634f, kAttnLn2 = 0.6931471805599453f;
constexpr int kTcRows = 128;                   // rows of an MMA
constexpr int kTcKeys = 128, kTcKeyShift = 7;  // keys of a tile

// The products below are called by a whole converged warp, and `lead` is nonzero in the one
// lane that issues them.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t lead;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(lead));
    return lead;
}
// Negates A of a product (an addend of its instruction descriptor).
constexpr uint32_t kNegateA = 1u << 13;
// A value that all lanes have, as one the compiler knows to be uniform: the products' operands
// then stay in uniform registers (else each product waits for moves there, 100 cycles instead
// of the 64 that a 128 x 128 x 16 one takes).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ int32_t uniform(int32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// D[128, N] (+)= A[128, 16] B[N, 16]^T, both operands in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, uint32_t acc)
{
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(id), "r"(acc), "r"(lead));
}
// The same with A in tensor memory: row r in lane r, two BF16 values of K a column.
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id,
                                       uint32_t acc)
{
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(id), "r"(acc), "r"(lead));
}
// Arrives on `mbar` when every product that the lane issued before has completed.
__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t* mbar)
{
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
            tc::smem_u32(mbar)), "r"(lead)
        : "memory");
}

// A bounded wait of a whole converged warp: it gives up for all lanes or for none, after
// which the role's waits return at once and it works no more.  Short, since the roles' code
// competes for the instruction cache.
struct WarpWait {
    volatile int32_t* abort;
    int32_t* status;
    bool gave_up;
    __device__ __forceinline__ WarpWait(int32_t* abort_flag, int32_t* status_word)
        : abort(abort_flag), status(status_word), gave_up(false) {}
    // times: of the limit of one wait, for one that others' whole tiles of rows pass in
    __device__ __forceinline__ void operator()(uint64_t* m, uint32_t parity, uint32_t times = 1)
    {
        if (__all_sync(0xffffffffu, mbar_test(m, parity))) return;
        uint32_t polls = 0, checks = 0;
        uint64_t since = 0;
        while (!gave_up && !tc::mbar_try_wait(m, parity)) {
            if (++polls % tc::kPollsPerCheck == 0) {
                const uint64_t now = tc::globaltimer_ns();
                if (since == 0) since = now;
                if (*abort || now - since > times * tc::kWaitLimitNs || ++checks > times * tc::kMaxTimerChecks) {
                    gave_up = true;
                    *abort = 1;
                    report_status(status, KDA_ERR_TIMEOUT);
                }
            }
        }
        gave_up = __any_sync(0xffffffffu, gave_up);
    }
    // A tile of rows takes a second at 10^8 keys.
    __device__ __forceinline__ void for_job(uint64_t* m, uint32_t parity) { (*this)(m, parity, 100); }
    // with the outcome of an earlier look (mbar_test): waits where it was too early
    __device__ __forceinline__ void after(bool seen, uint64_t* m, uint32_t parity)
    {
        if (!__all_sync(0xffffffffu, seen)) (*this)(m, parity);
    }
    __device__ __forceinline__ bool dead() const { return gave_up; }
};

// A role's place in a ring of N slots.
template <int N> struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// As tc::tmem_ld32, without the wait (tmem_ld_wait).
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, float* r)
{
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]),
          "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]),
          "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]),
          "=r"(u[31])
        : "r"(taddr)
        : "memory");
}
// The registers of the loads before it may be read after this; they pass through it, so that
// no use of them is moved ahead.
template <int N> __device__ __forceinline__ void tmem_ld_wait(float (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* u)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n" ::"r"(u[0]),
        "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
        "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]),
        "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]),
        "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]), "r"(u[29]),
        "r"(u[30]), "r"(u[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Stores a box of shared memory (swizzled as tma_load_3d leaves it) to a 3-D tensor map; the
// thread's stores are waited for together.
__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(tmap),
                 "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(src))
                 : "memory");
}
// The thread's stores so far have read shared memory (kRead), or are complete.
template <bool kRead> __device__ __forceinline__ void tma_store_wait()
{
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    if (kRead) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    else asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Brings a tensor map to where the copies look for it.
__device__ __forceinline__ void prefetch_map(const void* tmap)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(tmap) : "memory");
}

// Registers of a thread of the warps of this warpgroup from here on (all of whose warps call
// it), out of those that the block was launched with.
template <int N> __device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// ---------------------------------------------------------------- host
// [T, H, D] of 16-bit values, tokens `stride` elements apart, read as boxes of 64 channels of
// `heads` heads of `tokens` tokens in 128-byte swizzled rows (token, head); rows past the end
// read as zeros.
inline cudaError_t encode_heads(CUtensorMap* m, const void* base, int64_t T, int H, int D, int64_t stride, int heads,
                                int tokens)
{
    const EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A CTA's next tile of rows, from the warp that walks over them to the other roles.
struct AttnJob {
    AttnTile t;
    int32_t unit, piece, found;
};
// The CTA's round-th job of `jobs`, by a whole warp: to and fro over the CTAs, since the work
// falls from job to job.
__device__ __forceinline__ AttnJob attn_job(AttnWalk& walk, const AttnArgs& a, const AttnShape& sh, int32_t jobs,
                                            int32_t round)
{
    const int64_t at = (int64_t)round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    AttnJob job;
    job.found = 0;
    if (at < jobs) {
        const int32_t rest = a.splits > 1 ? (int32_t)at / a.splits : (int32_t)at;
        job.piece = (int32_t)at - rest * a.splits;
        job.unit = rest % sh.units;
        job.found = walk.next(a, rest / sh.units, job.t);
    }
    return job;
}

// Whether a kernel was given exactly the registers a thread that its setmaxnreg counts on:
// with fewer, the threads that ask for more would wait for good.
template <typename K> cudaError_t check_registers(K kern, int registers)
{
    cudaFuncAttributes f;
    const cudaError_t e = cudaFuncGetAttributes(&f, kern);
    if (e != cudaSuccess) return e;
    return f.numRegs == registers ? cudaSuccess : cudaErrorLaunchOutOfResources;
}

// Rows of a call cut into tiles of at most `rows`: as many heads of the group as fit and
// divide it, so that no tile has a head of another group.
inline AttnShape attn_shape(int32_t rows, int32_t Hq, int32_t Hk)
{
    AttnShape s;
    const int32_t G = Hq / Hk;
    s.heads = G < rows ? G : rows;
    while (G % s.heads != 0) --s.heads;
    s.parts = G / s.heads;
    s.tokens = rows / s.heads;
    s.units = Hk * s.parts;
    return s;
}
// Tiles of a call, at most: all but one of the sequences end in a tile of one token.
inline int64_t attn_tiles(int32_t N, int32_t T, int32_t tokens)
{
    return N < T ? (int64_t)(T - N) / tokens + N : T;
}
// Items of a kernel that starts a CTA a tile (attn_find).
inline int64_t attn_items(int32_t N, int32_t T, int32_t tokens)
{
    return N > kAttnOrdered ? (int64_t)T / tokens + N : attn_tiles(N, T, tokens);
}

}  // namespace kda
