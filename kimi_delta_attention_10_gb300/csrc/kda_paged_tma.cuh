// What the decode kernels share below their arithmetic: the walk over a CTA's rows,
// bounded waits, page lookups, TMA boxes and their tensor maps.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include <atomic>

#include "kda_paged_sched.cuh"
#include "kda_tc.cuh"

namespace kda {

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int x, int y,
                                            uint64_t* m)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(tc::smem_u32(m))
        : "memory");
}

__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// The rows (request, head unit) of a CTA's tiles, in order; every role walks its own.
struct DecodeWalk {
    int64_t pos, end, at;
    int32_t n, u, tile0, tile1, tiles, L;
    int32_t known;        // the request that L is of
    __device__ __forceinline__ explicit DecodeWalk(const DecodeRange& r)
        : pos(r.begin), end(r.end), at(r.at), n(r.n), u(0), tile0(0), tile1(0), tiles(0), L(r.L), known(r.n) {}
    // The next row with tiles tile0 .. tile1 - 1 (at least one) of this CTA.
    __device__ __forceinline__ bool next(const DecodeArgs& a, const DecodeShape& sh)
    {
        while (pos < end) {
            for (;; ++n) {
                if (n != known) {
                    L = decode_len(a, n);
                    known = n;
                }
                tiles = tiles_of(L, sh.tile_shift);
                const int64_t all = tiles ? (int64_t)(tiles + sh.start) * sh.units : 0;
                if (pos < at + all) break;
                at += all;
            }
            const int32_t places = tiles + sh.start;
            u = (int32_t)quotient(pos - at, places);
            const int64_t row = at + (int64_t)u * places;      // the row's first place
            tile0 = max((int32_t)(pos - row) - sh.start, 0);
            pos = min(end, row + places);
            tile1 = (int32_t)(pos - row) - sh.start;
            if (tile1 > tile0) return true;
        }
        return false;
    }
};

// Whether the phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* m, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(tc::smem_u32(m)), "r"(parity)
        : "memory");
    return ok != 0;
}

// A wait that gives up marks the CTA: its producer then stops, the other roles run
// their loops to the end without waiting or multiplying, so that all barriers meet.
struct BoundedWait {
    volatile int32_t* abort;
    int32_t* status;
    bool dead;
    __device__ __forceinline__ BoundedWait(int32_t* abort_flag, int32_t* status_word)
        : abort(abort_flag), status(status_word), dead(false) {}
    __device__ __forceinline__ void operator()(uint64_t* m, uint32_t parity)
    {
        if (dead) return;
        for (uint32_t j = 0; j < tc::kPollsPerCheck; ++j)
            if (tc::mbar_try_wait(m, parity)) return;
        const uint64_t t0 = tc::globaltimer_ns();
        for (uint32_t i = 0; i < tc::kMaxTimerChecks; ++i) {
            for (uint32_t j = 0; j < tc::kPollsPerCheck; ++j)
                if (tc::mbar_try_wait(m, parity)) return;
            if (*abort) break;
            if (tc::globaltimer_ns() - t0 > tc::kWaitLimitNs) break;
        }
        dead = true;
        *abort = 1;
        report_status(status, KDA_ERR_TIMEOUT);
    }
};

// The cache row (of num_pages * Hk * page_size) of a request's token `at` and head hk.
// An entry outside the cache is reported and read as page 0.
__device__ __forceinline__ int32_t page_row(const DecodeArgs& a, const int32_t* table, int hk, int at)
{
    int32_t page = table[at >> a.page_shift];
    if ((uint32_t)page >= (uint32_t)a.num_pages) {
        report_status(a.status, KDA_ERR_DEVICE_ARG);
        page = 0;
    }
    return ((page * a.Hk + hk) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
}

// ---------------------------------------------------------------- host
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_tiled()
{
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// rows x D values of a cache (or of q), read as boxes of box_rows x box_cols, swizzled
// in 128-byte rows or plain; rows past the end read as zeros.
inline cudaError_t encode_rows(CUtensorMap* m, const void* base, bool bf16, int64_t rows, int D,
                               int box_cols, int box_rows, bool swizzle)
{
    const EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)D * (bf16 ? 2 : 4)};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                          2, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Raises a kernel's dynamic shared memory, once per device: the setting stays with it.
template <typename K> cudaError_t allow_smem(K kern, uint32_t bytes, std::atomic<uint64_t>* set)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (set->load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) set->fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace kda
