// How the decode attention's work is dealt out, shared by its kernels and the join:
// every (request, head unit) row of `tiles` tiles lies on one axis of
// W = units * sum_n (tiles_n + start) places, ordered by request, unit, tile; each row
// begins with `start` places without a tile, which stand for the time that starting and
// ending a row costs.  CTA b of B = min(CTAs, W) takes W / B places, the first W % B CTAs
// one more.  A row whose tiles a CTA covers whole is finished there; of a split row
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

// A length that the table cannot hold counts as none.
__device__ __forceinline__ int32_t valid_len(const DecodeArgs& a, int32_t L)
{
    const int64_t most = (int64_t)a.max_pages << a.page_shift;
    return L < 0 || L > most ? 0 : L;
}
// Requests with a row.
__device__ __forceinline__ int32_t decode_requests(const DecodeArgs& a)
{
    return a.live == nullptr ? a.N : min(max(*a.live, 0), a.N);
}
__device__ __forceinline__ int32_t decode_len(const DecodeArgs& a, int32_t n)
{
    return valid_len(a, a.seq_lens[n]);
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
    int32_t n, L;         // request of place `begin`, and its length
};

__device__ __forceinline__ int32_t decode_places(const DecodeShape& s, int32_t L)
{
    const int32_t tiles = tiles_of(L, s.tile_shift);
    return tiles ? tiles + s.start : 0;                // an empty request has no row
}

// The CTAs' shares of W places.
struct DecodeShares {
    int64_t B, share, more;            // the first `more` CTAs of B take share + 1

    __device__ __forceinline__ DecodeShares(int64_t W, const DecodeShape& s)
    {
        B = W < s.ctas ? W : s.ctas;
        share = B ? quotient(W, B) : 0;
        more = W - share * B;
    }
    __device__ __forceinline__ int64_t begin(int64_t b) const { return b * share + min(b, more); }
    __device__ __forceinline__ int32_t cta_of(int64_t x) const
    {
        const int64_t edge = more * (share + 1);
        return (int32_t)(x < edge ? quotient(x, share + 1) : more + quotient(x - edge, share));
    }
};

// Leaves CTA b's split for the join (r.begin < r.end; else the CTA has none).
__device__ __forceinline__ void leave_split(const DecodeShape& s, const DecodeShares& shares, int32_t b,
                                            const DecodeRange& r, void* workspace)
{
    DecodeSplit split = {0, 0, 0, -1};
    if (r.begin < r.end) {
        const int32_t p = decode_places(s, r.L), u = (int32_t)quotient(r.begin - r.at, p);
        const int64_t tile = r.at + (int64_t)u * p + s.start, last = tile + p - s.start - 1;
        if (tile < r.begin && shares.cta_of(tile) + 1 == b)
            split = {r.n, u, b - 1, shares.cta_of(last)};
    }
    static_cast<DecodeSplit*>(workspace)[b] = split;
}

// Where the CTA's places lie: every warp works it out for itself from up to 4 requests a
// lane, loaded beforehand, so that the roles start without a barrier; with more requests
// the CTA's NT threads share them.  Warp 0 leaves the CTA's split, CTA 0 reports bad lengths.
constexpr int kLaneRequests = 4;
struct DecodeLens {
    int32_t L[kLaneRequests];          // of requests 4 lane .. 4 lane + 3, as given
    int32_t N;                         // requests with a row
    __device__ __forceinline__ void load(const DecodeArgs& a)
    {
        const int n0 = (threadIdx.x & 31) * kLaneRequests;
#pragma unroll
        for (int i = 0; i < kLaneRequests; ++i) L[i] = n0 + i < a.N ? a.seq_lens[n0 + i] : 0;
        N = decode_requests(a);
    }
};

__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

template <int NT>
__device__ __forceinline__ DecodeRange decode_range(const DecodeArgs& a, const DecodeShape& s,
                                                    const DecodeLens& lens, void* workspace)
{
    __shared__ int64_t sums[NT / 32];
    __shared__ DecodeRange range;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t b = blockIdx.x;
    DecodeRange r = {};
    if (a.N <= 32 * kLaneRequests) {
        int32_t L[kLaneRequests];
        int64_t mine = 0;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kLaneRequests; ++i) {
            const int32_t given = lane * kLaneRequests + i < lens.N ? lens.L[i] : 0;
            L[i] = valid_len(a, given);
            bad |= L[i] != given;
            mine += decode_places(s, L[i]);
        }
        const int64_t upto = warp_scan(mine, lane);
        const DecodeShares shares(__shfl_sync(0xffffffffu, upto, 31) * s.units, s);
        if (b < shares.B) {
            r.begin = shares.begin(b);
            r.end = shares.begin(b + 1);
            const int owner = __ffs(__ballot_sync(0xffffffffu, r.begin < upto * s.units)) - 1;
            int64_t at = upto - mine;
            int32_t n = lane * kLaneRequests, len = L[0];
            bool found = false;
#pragma unroll
            for (int i = 0; i < kLaneRequests; ++i) {
                const int64_t next = at + decode_places(s, L[i]);
                if (!found) {
                    found = r.begin < next * s.units;
                    if (found) {
                        n = lane * kLaneRequests + i;
                        len = L[i];
                    } else {
                        at = next;
                    }
                }
            }
            r.n = __shfl_sync(0xffffffffu, n, owner);
            r.L = __shfl_sync(0xffffffffu, len, owner);
            r.at = __shfl_sync(0xffffffffu, at, owner) * s.units;
        }
        if (tid == 0) leave_split(s, shares, b, r, workspace);
        if (b == 0 && warp == 0 && bad) report_status(a.status, KDA_ERR_DEVICE_ARG);
        return r;
    }
    const int32_t N = decode_requests(a), per = (N + NT - 1) / NT;      // consecutive requests per thread
    const int32_t n0 = min(tid * per, N), n1 = min(n0 + per, N);
    int64_t mine = 0;
    for (int32_t n = n0; n < n1; ++n) mine += decode_places(s, decode_len(a, n));
    int64_t upto = warp_scan(mine, lane);
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int64_t total = 0, before = upto - mine;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    const DecodeShares shares(total * s.units, s);
    if (b < shares.B) {
        r.begin = shares.begin(b);
        r.end = shares.begin(b + 1);
        if (before * s.units <= r.begin && r.begin < (before + mine) * s.units) {
            int64_t at = before;
            for (r.n = n0;; ++r.n) {
                r.L = decode_len(a, r.n);
                const int64_t next = at + decode_places(s, r.L);
                if (r.begin < next * s.units) break;
                at = next;
            }
            r.at = at * s.units;
            range = r;
            leave_split(s, shares, b, r, workspace);
        }
    } else if (tid == 0) {
        range = r;
        leave_split(s, shares, b, r, workspace);
    }
    if (b == 0)
        for (int32_t n = n0; n < n1; ++n)
            if (a.seq_lens[n] != decode_len(a, n)) report_status(a.status, KDA_ERR_DEVICE_ARG);
    __syncthreads();
    return range;
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
