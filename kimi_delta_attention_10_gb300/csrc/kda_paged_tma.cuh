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

// The rows (request, head unit) of a CTA's tiles, in order; every role walks its own.  A
// role is one warp or thread, whose time per row is its instructions' latency: one
// division at the start, none after it, and the next request's length loaded ahead.
struct DecodeWalk {
    int64_t left;         // places still to come
    int32_t skip;         // places of the next row that are an earlier CTA's
    int32_t n, L, tiles;  // the request, its length and tiles
    int32_t ahead;        // length of request n + 1, as given
    int32_t hk, part;     // head unit: key-value head, part of its group of query heads
    int32_t tile0, tile1;
    int32_t parts;        // units per key-value head
    __device__ __forceinline__ DecodeWalk(const DecodeRange& r, const DecodeArgs& a, const DecodeShape& sh,
                                          int32_t units_per_head)
        : left(r.end - r.begin), skip(0), n(r.n), L(r.L), tiles(tiles_of(r.L, sh.tile_shift)), ahead(0),
          hk(0), part(-1), tile0(0), tile1(0), parts(units_per_head)
    {
        if (left <= 0) return;
        const int32_t places = tiles + sh.start;
        const int32_t u = (int32_t)quotient(r.begin - r.at, places);
        skip = (int32_t)(r.begin - r.at - (int64_t)u * places);
        hk = u / parts;
        part = u - hk * parts - 1;
        if (n + 1 < a.N) ahead = a.seq_lens[n + 1];
    }
    // The next row with tiles tile0 .. tile1 - 1 (at least one) of this CTA.
    __device__ __forceinline__ bool next(const DecodeArgs& a, const DecodeShape& sh)
    {
        while (left > 0) {
            if (++part == parts) {
                part = 0;
                if (++hk == a.Hk) {
                    hk = 0;
                    do {
                        if (++n >= a.N) return false;      // lengths that changed meanwhile
                        L = valid_len(a, ahead);
                        tiles = tiles_of(L, sh.tile_shift);
                        if (n + 1 < a.N) ahead = a.seq_lens[n + 1];
                    } while (tiles == 0);
                }
            }
            const int32_t places = tiles + sh.start - skip;
            const int32_t take = left < places ? (int32_t)left : places;
            tile0 = max(skip - sh.start, 0);
            tile1 = skip + take - sh.start;
            left -= take;
            skip = 0;
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

// The cache row (of num_pages * Hk * page_size) of head hk's token `at`, with the block
// table's entry for it.  An entry outside the cache is reported and read as page 0.
__device__ __forceinline__ int32_t page_row(const DecodeArgs& a, int32_t page, int hk, int at)
{
    if ((uint32_t)page >= (uint32_t)a.num_pages) {
        report_status(a.status, KDA_ERR_DEVICE_ARG);
        page = 0;
    }
    return ((page * a.Hk + hk) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
}

// A producer's tiles in order.  The table's entries are asked for before the wait for the
// tile's slot, and looked at after it.
struct DecodeTile {
    int32_t boxes;        // boxes of the tile; this lane has one if its `token` is within
    int32_t entry;        // the block table's, for the lane's box
    int32_t hk, at;       // head, and the token at which the lane's box begins
    int32_t n, part;      // the row, for its queries
    bool opens;           // the row's first tile here
    // lane_token: where in a tile the lane's box begins; a box holds 1 << shift tokens
    __device__ __forceinline__ bool next(DecodeWalk& w, int& t, const DecodeArgs& a, const DecodeShape& sh,
                                         int tile, int shift, int lane_token)
    {
        opens = ++t >= w.tile1;
        if (opens) {
            if (!w.next(a, sh)) return false;
            t = w.tile0;
        }
        const int tok = t * tile;
        boxes = (min(tile, w.L - tok) + (1 << shift) - 1) >> shift;
        at = tok + lane_token;
        hk = w.hk;
        n = w.n;
        part = w.part;
        entry = 0;
        if (lane_token < boxes << shift) entry = a.table[(int64_t)n * a.max_pages + (at >> a.page_shift)];
        return true;
    }
};

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
