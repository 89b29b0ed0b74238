// How the decode attention's work is dealt out, shared by its kernels and the join:
// every (request, head unit) row of `tiles` tiles lies on one axis of
// W = units * sum_n (tiles_n + start) places, ordered by request, unit, tile; each row
// begins with `start` places without a tile, which stand for the time that starting and
// ending a row costs.  CTA b of B = min(CTAs, W) takes W / B places, the first W % B
// CTAs one more.  A row whose tiles a CTA covers whole is finished there; of a split row
// each CTA leaves a piece (maximum, sum, unscaled output) in one of its two slots: slot
// 2 b where the row's tiles began before the CTA's, 2 b + 1 where they begin in them.
// A CTA has at most one of each.
#pragma once

#include <stdint.h>

#include "kda_paged.cuh"

namespace kda {

struct DecodeShape {
    int32_t units;        // head units per request
    int32_t heads;        // query heads per unit (the last of a group may have fewer)
    int32_t ctas;         // CTAs launched
    int32_t tile_shift;   // log2 of the tokens per tile
    int32_t start;        // places without a tile at the beginning of a row
};



// The split row that a CTA's tiles begin inside of, for the join: its request and unit,
// and the CTAs of its first and last tile (last < first: none, or not its first split).
struct alignas(16) DecodeSplit {
    int32_t n, u, first, last;
};

// Workspace: the CTAs' splits, then the pieces' (m, l) pairs [2 CTAs][heads], then
// their outputs [2 CTAs][heads][D].
__host__ __device__ inline int64_t decode_ml_offset(const DecodeShape& s)
{
    return ((int64_t)s.ctas * sizeof(DecodeSplit) + 255) / 256 * 256;
}
__host__ __device__ inline int64_t decode_o_offset(const DecodeShape& s)
{
    return decode_ml_offset(s) + ((int64_t)2 * s.ctas * s.heads * 8 + 255) / 256 * 256;
}
inline int64_t decode_workspace(const DecodeShape& s, int32_t D)
{
    return decode_o_offset(s) + (int64_t)2 * s.ctas * s.heads * D * 4;
}

__device__ __forceinline__ int32_t decode_len(const DecodeArgs& a, int32_t n)
{
    const int32_t L = a.seq_lens[n];
    const int64_t most = (int64_t)a.max_pages << a.page_shift;
    return L < 0 || L > most ? 0 : L;
}

__device__ __forceinline__ int32_t tiles_of(int32_t L, int shift)
{
    return (int32_t)(((int64_t)L + (1 << shift) - 1) >> shift);
}

// a / b for a >= 0, b > 0; the 64-bit division is a call of a hundred instructions.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

struct DecodeRange {
    int64_t begin, end;   // the CTA's places
    int64_t at;           // places of the requests before `n`, all units
    int32_t n;            // request of place `begin`
};

// Called by NT threads of a CTA (a multiple of 32): where the CTA's places lie.  It also
// leaves the CTA's split for the join; CTA 0 reports bad lengths.
template <int NT>
__device__ __forceinline__ DecodeRange decode_range(const DecodeArgs& a, const DecodeShape& s,
                                                    void* workspace)
{
    __shared__ int64_t sums[NT / 32];
    __shared__ DecodeRange range;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t per = (a.N + NT - 1) / NT;         // consecutive requests per thread
    const int32_t n0 = min(tid * per, a.N), n1 = min(n0 + per, a.N);
    auto places = [&](int32_t n) {
        const int32_t tiles = tiles_of(decode_len(a, n), s.tile_shift);
        return tiles ? tiles + s.start : 0;           // an empty request has no row
    };
    int64_t mine = 0;
    for (int32_t n = n0; n < n1; ++n) mine += places(n);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int64_t total = 0, before = upto - mine;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    const int64_t W = total * s.units, b = blockIdx.x;
    const int64_t B = W < s.ctas ? W : s.ctas;
    int64_t begin = 0, end = 0;
    if (b < B) {
        const int64_t share = quotient(W, B), more = W - share * B;
        begin = b * share + min(b, more);
        end = begin + share + (b < more);
        if (before * s.units <= begin && begin < (before + mine) * s.units) {
            int64_t at = before;
            int32_t n = n0;
            for (;; ++n) {
                const int64_t next = at + places(n);
                if (begin < next * s.units) break;
                at = next;
            }
            range.n = n;
            range.at = at * s.units;
            // the row of place `begin`, and the CTAs of its first and last tile
            const int32_t p = places(n);
            const int32_t u = (int32_t)quotient(begin - range.at, p);
            const int64_t tile = range.at + (int64_t)u * p + s.start, last = tile + p - s.start - 1;
            auto cta_of = [&](int64_t x) {
                const int64_t edge = more * (share + 1);
                return (int32_t)(x < edge ? quotient(x, share + 1) : more + quotient(x - edge, share));
            };
            DecodeSplit split = {n, u, 0, -1};
            if (tile < begin && cta_of(tile) + 1 == b) {
                split.first = (int32_t)b - 1;
                split.last = cta_of(last);
            }
            static_cast<DecodeSplit*>(workspace)[b] = split;
        }
    } else if (tid == 0) {
        static_cast<DecodeSplit*>(workspace)[b] = {0, 0, 0, -1};
    }
    if (b == 0)
        for (int32_t n = n0; n < n1; ++n)
            if (a.seq_lens[n] != decode_len(a, n)) report_status(a.status, KDA_ERR_DEVICE_ARG);
    __syncthreads();
    DecodeRange r = range;
    r.begin = begin;
    r.end = end;
    return r;
}

// Joins the split rows and writes the rows of empty requests.
cudaError_t launch_decode_join(const DecodeArgs& a, const DecodeShape& s, cudaStream_t stream);

// The tensor-core kernel (BF16).
DecodeShape decode_tc_shape(const DecodeArgs& a);
cudaError_t launch_paged_decode_tc(const DecodeArgs& a, const DecodeShape& s, cudaStream_t stream);

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T>
__device__ __forceinline__ void store_one(T* p, float x);
template <>
__device__ __forceinline__ void store_one<float>(float* p, float x)
{
    *p = x;
}
template <>
__device__ __forceinline__ void store_one<__nv_bfloat16>(__nv_bfloat16* p, float x)
{
    *p = __float2bfloat16_rn(x);
}

}  // namespace kda
