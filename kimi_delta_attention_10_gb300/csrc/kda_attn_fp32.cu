// Attention for several tokens a sequence on CUDA cores (IEEE FP32 products): forward
// over packed or paged keys, its backward, and the join of pieces of the keys' axis for
// either type.
//
//     s_ij = scale q_i . k_j,  lse_i = log sum_j e^(s_ij),  o_i = sum_j e^(s_ij - lse_i) v_j
//     p_ij = e^(s_ij - lse_i), delta_i = do_i . o_i, ds_ij = p_ij (do_i . v_j - delta_i)
//     dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//
// Bound by the FMA pipe: 4 D operations a score forward, 14 D backward (the two backward
// kernels each form the scores and the products with v again, so that dk and dv are summed
// in one CTA over all heads of the group and dq in another: no atomics, the same bits in
// every run).  A CTA of 256 threads holds a tile of scores in registers, up to 8 x 4 a
// thread; operands are read from shared memory four channels at a time, the rows of a
// tile padded by 16 bytes so that 16 lanes' rows lie in different banks.
//
// Measured: 2048 tokens, 16 heads of 64 channels, 244 us (35 TFLOP/s, 47% of the FMA pipe's
// peak; it is busy 55% of the cycles: two warps a scheduler wait for their own instructions,
// and twice as many with smaller tiles read more); forward and backward of 1024 tokens 327 us:
// 92 in three pieces and 9 for their join, delta 4, dk and dv 137, dq 111.  The last two walk over 16
// tiles at most, 14.3 on the mean SM, in 8.6 and 6.9 us a step whose products would take 4.3
// and 3.2 at the pipe's peak: eight warps go through scores, weights and sums together.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include <atomic>

#include "kda_attn_tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kThreads = 256;
constexpr int kKeys = 64, kKeyShift = 6;       // keys of a tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x)
{
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}

// A tile's rows: row r is token r / heads of the tile, head first + r % heads of the group.
struct RowMap {
    int32_t heads, rows;     // heads of the tile (a row's divisor), rows in use
    int32_t row0, head0;     // first packed token, first query head
    __device__ __forceinline__ RowMap(const AttnShape& sh, int32_t unit, int32_t token0, int32_t tokens)
        : heads(sh.heads), rows(tokens * sh.heads), row0(token0), head0(unit * sh.heads) {}
    // (token, head) of row r; false: the row is not in use
    __device__ __forceinline__ bool at(int32_t r, int32_t& token, int32_t& head) const
    {
        const int32_t i = r / heads, g = r - i * heads;
        token = row0 + i;
        head = head0 + g;
        return r < rows;
    }
};

// ROWS rows of D values to shared memory rows of D + 4, zeros where a row is not in use.
template <int ROWS, int D>
__device__ __forceinline__ void load_rows(float* dst, const float* x, int64_t stride, const RowMap& m)
{
    for (int e = threadIdx.x; e < ROWS * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        int32_t token, head;
        const bool ok = m.at(r, token, head);
        cp_async16(dst + r * (D + 4) + c, ok ? x + token * stride + (int64_t)head * D + c : x, ok);
    }
}
// Keys or values `at` .. at + 63 of head hk, zeros past `end`.
template <int D, int PITCH>
__device__ __forceinline__ void load_keys(float* dst, const AttnArgs& a, const float* x, int64_t stride,
                                          const AttnTile& t, int32_t hk, int32_t at, int32_t end)
{
    for (int e = threadIdx.x; e < kKeys * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = e % (D / 4) * 4, j = at + r;
        const bool ok = j < end;
        const float* src = x;
        if (ok)
            src = a.table != nullptr ? x + attn_page_row(a, t.n, hk, j) * D + c
                                     : x + (t.seq0 + j) * stride + (int64_t)hk * D + c;
        cp_async16(dst + r * PITCH + c, src, ok);
    }
}

// s[i][c] = sum over channels of A row (ty * R + i) and B row (tx + 16 c).
template <int R, int D>
__device__ __forceinline__ void scores(float (&s)[R][4], const float* A, const float* B, int ty, int tx)
{
    float2 acc[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 x[R], y[4];
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const float4*>(A + (ty * R + i) * (D + 4) + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const float4*>(B + (tx + 16 * c) * (D + 4) + d);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[i][c] = fma2(make_float2(x[i].x, x[i].y), make_float2(y[c].x, y[c].y), acc[i][c]);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[i][c] = fma2(make_float2(x[i].z, x[i].w), make_float2(y[c].z, y[c].w), acc[i][c]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[i][c] = acc[i][c].x + acc[i][c].y;
}

// o[i][h] (four channels 4 tx + 64 h of row ty * R + i) += sum over `keys` of
// w[row][key] x[key][channel]; w in rows of `pitch`.
template <int R, int H, int PITCH>
__device__ __forceinline__ void accumulate(float2 (&o)[R][2 * H], const float* w, int pitch, const float* x,
                                           int ty, int tx)
{
#pragma unroll 2
    for (int j = 0; j < kKeys; j += 4) {
        float4 p[R];
#pragma unroll
        for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4*>(w + (ty * R + i) * pitch + j);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float4 y = *reinterpret_cast<const float4*>(x + (j + k) * PITCH + 4 * tx + 64 * h);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float2 pk = both(k == 0 ? p[i].x : k == 1 ? p[i].y : k == 2 ? p[i].z : p[i].w);
                    o[i][2 * h] = fma2(pk, make_float2(y.x, y.y), o[i][2 * h]);
                    o[i][2 * h + 1] = fma2(pk, make_float2(y.z, y.w), o[i][2 * h + 1]);
                }
            }
        }
    }
}
// The same with w transposed, of eight keys a thread: o of key 8 ty + i += sum over rows of
// w[row][key] x[row][channel]; w single, in rows of `pitch`.
template <int ROWS, int H, int PITCH>
__device__ __forceinline__ void accumulate_t(float2 (&o)[8][2 * H], const float* w, int pitch, const float* x,
                                             int ty, int tx)
{
#pragma unroll 4
    for (int r = 0; r < ROWS; ++r) {
        const float4 p = *reinterpret_cast<const float4*>(w + r * pitch + 8 * ty),
                     q = *reinterpret_cast<const float4*>(w + r * pitch + 8 * ty + 4);
        const float2 pk[8] = {both(p.x), both(p.y), both(p.z), both(p.w), both(q.x), both(q.y), both(q.z), both(q.w)};
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const float4 y = *reinterpret_cast<const float4*>(x + r * PITCH + 4 * tx + 64 * h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i][2 * h] = fma2(pk[i], make_float2(y.x, y.y), o[i][2 * h]);
                o[i][2 * h + 1] = fma2(pk[i], make_float2(y.z, y.w), o[i][2 * h + 1]);
            }
        }
    }
}

__device__ __forceinline__ float over16(float x, bool sum)
{
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        x = sum ? x + y : fmaxf(x, y);
    }
    return x;
}

// ---------------------------------------------------------------- forward
// A tile of 16 R rows: the fewer rows a call has, the smaller, down to one row a thread.
template <int D, int R> struct Fwd {
    static constexpr int ROWS = 16 * R;
    static constexpr int OFF_K = ROWS * (D + 4), OFF_V = OFF_K + kKeys * (D + 4), OFF_P = OFF_V + kKeys * D;
    static constexpr int PITCH_P = kKeys + 4;
    static constexpr uint32_t SMEM = (OFF_P + ROWS * PITCH_P) * 4;
    static constexpr int CTAS = R <= 2 || (R == 4 && D == 64) ? 2 : 1;         // per SM
    static_assert(CTAS * (SMEM + 1024 + 64) <= 228 * 1024, "shared memory of an SM");
};

template <int D, int R>
__global__ void __launch_bounds__(kThreads, (Fwd<D, R>::CTAS)) attn_fwd_kernel(AttnArgs a, AttnShape sh)
{
    using F = Fwd<D, R>;
    constexpr int H = D / 64;
    extern __shared__ __align__(16) float sm[];
    __shared__ AttnTile s_tile;
    __shared__ int s_found;
    float *sQ = sm, *sK = sm + F::OFF_K, *sV = sm + F::OFF_V, *sP = sm + F::OFF_P;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    wait_for_previous();
    const int32_t piece = blockIdx.x % a.splits, unit = blockIdx.x / a.splits % sh.units,
                  item = blockIdx.x / a.splits / sh.units;
    const bool bad = a.N > kAttnOrdered && attn_bad(a);
    if (tid < 32) {
        AttnTile t;
        const bool found = attn_find(a, bad, item, sh.tokens, kKeyShift, t);
        if (tid == 0) {
            s_tile = t;
            s_found = found;
            if (blockIdx.x == 0 && a.pieces > 1)
                *static_cast<int32_t*>(a.workspace) = (a.N > kAttnOrdered ? !bad : found) ? a.cu[a.N] : 0;
        }
    }
    __syncthreads();
    if (!s_found) return;
    const AttnTile t = s_tile;
    const int32_t hk = unit / sh.parts;
    const RowMap rows(sh, unit, t.row0, t.tokens);
    const float *q = static_cast<const float*>(a.q), *k = static_cast<const float*>(a.k), *v = static_cast<const float*>(a.v);
    const int32_t keys = attn_keys(a, t), tiles = (keys + kKeys - 1) / kKeys;
    const int32_t j0 = (int32_t)((int64_t)tiles * piece / a.splits),
                  j1 = (int32_t)((int64_t)tiles * (piece + 1) / a.splits);
    const float c = a.scale * kLog2e;

    int32_t limit[R];                          // keys that each of the thread's rows sees
    float m[R], l[R];
    float2 o[R][2 * H];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        limit[i] = a.causal ? t.pos0 + (ty * R + i) / sh.heads + 1 : t.kv_len;
        m[i] = -CUDART_INF_F;
        l[i] = 0.f;
#pragma unroll
        for (int h = 0; h < 2 * H; ++h) o[i][h] = make_float2(0.f, 0.f);
    }
    if (j0 < j1) {
        load_rows<F::ROWS, D>(sQ, q, a.q_stride, rows);
        load_keys<D, D + 4>(sK, a, k, a.k_stride, t, hk, j0 * kKeys, keys);
        cp_async_commit();
        load_keys<D, D>(sV, a, v, a.v_stride, t, hk, j0 * kKeys, keys);
        cp_async_commit();
    }
    for (int32_t j = j0; j < j1; ++j) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        float s[R][4];
        scores<R, D>(s, sQ, sK, ty, tx);
        __syncthreads();
        if (j + 1 < j1) load_keys<D, D + 4>(sK, a, k, a.k_stride, t, hk, (j + 1) * kKeys, keys);
        cp_async_commit();
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float top = -CUDART_INF_F;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                s[i][n] = j * kKeys + tx + 16 * n < limit[i] ? s[i][n] * c : -CUDART_INF_F;
                top = fmaxf(top, s[i][n]);
            }
            top = fmaxf(m[i], over16(top, false));
            const float ref = top == -CUDART_INF_F ? 0.f : top, keep = exp2f(m[i] - ref);
            m[i] = top;
            l[i] *= keep;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float e = exp2f(s[i][n] - ref);
                l[i] += e;
                sP[(ty * R + i) * F::PITCH_P + tx + 16 * n] = e;
            }
#pragma unroll
            for (int h = 0; h < 2 * H; ++h) o[i][h] = mul2(o[i][h], both(keep));
        }
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        accumulate<R, H, D>(o, sP, F::PITCH_P, sV, ty, tx);
        __syncthreads();
        if (j + 1 < j1) load_keys<D, D>(sV, a, v, a.v_stride, t, hk, (j + 1) * kKeys, keys);
        cp_async_commit();
    }
    char* ws = static_cast<char*>(a.workspace);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float sum = over16(l[i], true), inv = sum == 0.f ? 0.f : 1.f / sum;
        const float ref = m[i] == -CUDART_INF_F ? 0.f : m[i];
        int32_t token, head;
        if (!rows.at(ty * R + i, token, head)) continue;
        const int64_t r = (int64_t)token * a.Hq + head;
        const float lse = ref * kLn2 + logf(sum);
        if (a.pieces > 1) {
            float* y = reinterpret_cast<float*>(ws + attn_pieces_o(a, piece)) + r * D + 4 * tx;
            if (tx == 0) reinterpret_cast<float*>(ws + attn_pieces_lse(a, piece))[r] = lse;
#pragma unroll
            for (int h = 0; h < H; ++h)
                store4(y + 64 * h, make_float4(o[i][2 * h].x * inv, o[i][2 * h].y * inv, o[i][2 * h + 1].x * inv,
                                               o[i][2 * h + 1].y * inv));
        } else {
            float* y = static_cast<float*>(a.out) + r * D + 4 * tx;
            if (tx == 0 && a.lse != nullptr) a.lse[r] = lse;
#pragma unroll
            for (int h = 0; h < H; ++h)
                store4(y + 64 * h, make_float4(o[i][2 * h].x * inv, o[i][2 * h].y * inv, o[i][2 * h + 1].x * inv,
                                               o[i][2 * h + 1].y * inv));
        }
    }
}

// ---------------------------------------------------------------- join
// out = sum_p e^(lse_p - lse) o_p, lse = log sum_p e^(lse_p): a warp a row, whose lanes have D / 32
// channels each.  A piece without weight (lse -infinity) is not read.
template <typename T, int D> __global__ void __launch_bounds__(256) attn_join_kernel(AttnArgs a)
{
    constexpr int C = D / 32;
    wait_for_previous();
    const char* ws = static_cast<const char*>(a.workspace);
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (int64_t)*reinterpret_cast<const int32_t*>(ws) * a.Hq) return;
    float top = -CUDART_INF_F;
    bool nan = false;
    for (int p = lane; p < a.pieces; p += 32) {
        const float x = reinterpret_cast<const float*>(ws + attn_pieces_lse(a, p))[row];
        top = fmaxf(top, x);
        nan |= x != x;
    }
    top = warp_max(top);
    nan = __any_sync(0xffffffffu, nan);
    // the pieces' outputs are asked for four at a time, and one without weight is not used
    float sum = 0.f, o[C] = {};
    for (int p0 = 0; p0 < a.pieces; p0 += 4) {
        float w[4], z[4][C];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int p = min(p0 + k, a.pieces - 1);
            w[k] = reinterpret_cast<const float*>(ws + attn_pieces_lse(a, p))[row];
            const float* y = reinterpret_cast<const float*>(ws + attn_pieces_o(a, p)) + row * D + C * lane;
            if constexpr (C == 4) *reinterpret_cast<float4*>(z[k]) = *reinterpret_cast<const float4*>(y);
            else *reinterpret_cast<float2*>(z[k]) = *reinterpret_cast<const float2*>(y);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (p0 + k >= a.pieces || w[k] == -CUDART_INF_F) continue;
            const float x = exp2f((w[k] - top) * kLog2e);
            sum += x;
#pragma unroll
            for (int i = 0; i < C; ++i) o[i] = fmaf(x, z[k][i], o[i]);
        }
    }
    const float inv = nan ? CUDART_NAN_F : sum == 0.f ? 0.f : 1.f / sum;
    if (lane == 0 && a.lse != nullptr)
        a.lse[row] = nan ? CUDART_NAN_F : sum == 0.f ? -CUDART_INF_F : top + logf(sum);
    T* y = static_cast<T*>(a.out) + row * D + C * lane;
    if constexpr (C == 4) {
        store4(y, make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv));
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float2*>(y) = make_float2(o[0] * inv, o[1] * inv);
    } else {
        *reinterpret_cast<uint32_t*>(y) = pack_bf16(o[0] * inv, o[1] * inv);
    }
}

// ---------------------------------------------------------------- backward
__device__ __forceinline__ float dot16(const uint4& x, const uint4& y, float)
{
    const float4 *a = reinterpret_cast<const float4*>(&x), *b = reinterpret_cast<const float4*>(&y);
    return fmaf(a->x, b->x, fmaf(a->y, b->y, fmaf(a->z, b->z, a->w * b->w)));
}
__device__ __forceinline__ float dot16(const uint4& x, const uint4& y, __nv_bfloat16)
{
    const uint32_t *a = &x.x, *b = &y.x;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), s);
        s = fmaf(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(b[i] & 0xffff0000u), s);
    }
    return s;
}
// delta = do . o of every row: 16 bytes a lane, kDeltaRows times as many rows as a warp's lanes
// cover in flight (HBM-bound).
constexpr int kDeltaRows = 4;
template <typename T, int D> struct Delta {
    static constexpr int LANES = D * sizeof(T) / 16, PER_WARP = 32 / LANES * kDeltaRows;
    static constexpr int PER_BLOCK = 8 * PER_WARP;
};
template <typename T, int D> __global__ void __launch_bounds__(256) attn_delta_kernel(AttnArgs a)
{
    using C = Delta<T, D>;
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.T * a.Hq;
    const int64_t row0 = (int64_t)blockIdx.x * C::PER_BLOCK + (threadIdx.x >> 5) * C::PER_WARP + lane / C::LANES;
    uint4 x[kDeltaRows], y[kDeltaRows];
#pragma unroll
    for (int k = 0; k < kDeltaRows; ++k) {
        const int64_t r = min(row0 + k * (32 / C::LANES), rows - 1) * C::LANES + lane % C::LANES;
        x[k] = static_cast<const uint4*>(a.dout)[r];
        y[k] = static_cast<const uint4*>(a.out)[r];
    }
#pragma unroll
    for (int k = 0; k < kDeltaRows; ++k) {
        float s = dot16(x[k], y[k], T());
#pragma unroll
        for (int o = C::LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const int64_t r = row0 + k * (32 / C::LANES);
        if (lane % C::LANES == 0 && r < rows) a.delta[r] = s;
    }
}

constexpr int kBwdRows = 64;                   // rows of a backward tile

// The two tiles that a CTA keeps (keys and values, or queries and dO), and one or, where
// shared memory has room, two stages of the two that it walks over.
template <int D> struct Bwd {
    static constexpr int STAGES = D == 64 ? 2 : 1;
    static constexpr int TILE = 64 * (D + 4), PITCH_P = kKeys + 4, STATS = 3 * kBwdRows;
    static constexpr int OFF_WALK = 2 * TILE, OFF_P = OFF_WALK + STAGES * 2 * TILE,
                         OFF_DS = OFF_P + kBwdRows * PITCH_P, OFF_L = OFF_DS + kBwdRows * PITCH_P;
    static constexpr uint32_t SMEM = (OFF_L + STAGES * STATS) * 4;
};

// lse and delta of a tile's rows, copied beside the tile, and how many keys each sees: of `end`,
// the first token's pos0 + 1 on.  A row that is not in use sees none: its zeros times a key with an
// infinity are NaN.
__device__ __forceinline__ void load_stats(float* dst, const AttnArgs& a, const RowMap& rows, int32_t pos0,
                                           int32_t end)
{
    const int r = threadIdx.x;
    if (r >= kBwdRows) return;
    int32_t token, head;
    const bool used = rows.at(r, token, head);
    reinterpret_cast<int32_t*>(dst)[2 * kBwdRows + r] = used ? min(end, pos0 + token - rows.row0 + 1) : 0;
    if (used) {
        const int64_t at = (int64_t)token * a.Hq + head;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst + r)), "l"(a.lse_in + at) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst + kBwdRows + r)), "l"(a.delta + at)
                     : "memory");
    } else {
        dst[r] = CUDART_INF_F;
        dst[kBwdRows + r] = 0.f;
    }
}

// P and dS of a tile: rows ty * 4 + i, keys tx + 16 n.
template <int D>
__device__ __forceinline__ void weights(float (&p)[4][4], float (&ds)[4][4], const float* q, const float* dout,
                                        const float* k, const float* v, const float* stats, const AttnArgs& a,
                                        int32_t key0, int ty, int tx)
{
    const float c = a.scale * kLog2e;
    scores<4, D>(p, q, k, ty, tx);
    scores<4, D>(ds, dout, v, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        const int32_t limit = reinterpret_cast<const int32_t*>(stats)[2 * kBwdRows + r];
        // a row without weight (lse -infinity) gives none
        const float lse = stats[r] == -CUDART_INF_F ? CUDART_INF_F : stats[r] * kLog2e, delta = stats[kBwdRows + r];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const bool live = key0 + tx + 16 * n < limit;
            p[i][n] = live ? exp2f(fmaf(p[i][n], c, -lse)) : 0.f;
            ds[i][n] = live ? p[i][n] * (ds[i][n] - delta) : 0.f;
        }
    }
}

// Waits for the copies of a tile, those of the next one (if any) still under way.
template <int STAGES> __device__ __forceinline__ void landed()
{
    if (STAGES == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else cp_async_wait_all();
    __syncthreads();
}

// dk and dv of 64 keys, over all rows that see them.
template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_bwd_kv_kernel(AttnArgs a, AttnShape sh)
{
    using B = Bwd<D>;
    constexpr int H = D / 64;
    extern __shared__ __align__(16) float sm[];
    __shared__ AttnTile s_tile;
    __shared__ int s_found;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    wait_for_previous();
    const int32_t hk = blockIdx.x % a.Hk, item = blockIdx.x / a.Hk;
    const bool bad = a.N > kAttnOrdered && attn_bad(a);
    if (tid < 32) {
        AttnTile t;
        const bool found = attn_find(a, bad, item, kKeys, kKeyShift, t);
        if (tid == 0) {
            s_tile = t;
            s_found = found;
        }
    }
    __syncthreads();
    if (!s_found) return;
    const AttnTile t = s_tile;
    // the tile found has t.index tiles of queries before it; the one with as many behind it
    const int32_t nt = (t.seq_tokens + kKeys - 1) / kKeys, key0 = (nt - 1 - t.index) * kKeys;
    const int32_t end = t.seq_tokens;
    const int32_t left = end - key0, per = (left + sh.tokens - 1) / sh.tokens, n = per * sh.parts;
    load_keys<D, D + 4>(sm, a, static_cast<const float*>(a.k), a.k_stride, t, hk, key0, end);
    load_keys<D, D + 4>(sm + B::TILE, a, static_cast<const float*>(a.v), a.v_stride, t, hk, key0, end);
    auto walked = [&](int32_t i) { return sm + B::OFF_WALK + i % B::STAGES * 2 * B::TILE; };
    auto stats = [&](int32_t i) { return sm + B::OFF_L + i % B::STAGES * B::STATS; };
    auto load = [&](int32_t i) {
        if (i < n) {
            const int32_t part = i / per, at = key0 + (i - part * per) * sh.tokens;
            const RowMap rows(sh, hk * sh.parts + part, t.seq0 + at, min(sh.tokens, end - at));
            load_rows<kBwdRows, D>(walked(i), static_cast<const float*>(a.q), a.q_stride, rows);
            load_rows<kBwdRows, D>(walked(i) + B::TILE, static_cast<const float*>(a.dout), (int64_t)a.Hq * D, rows);
            load_stats(stats(i), a, rows, at, end);
        }
        cp_async_commit();
    };
    // half of the threads add up dv, the others dk: eight keys and 4 H channels each
    const bool keys = tid >= kThreads / 2;
    const int gy = (tid & (kThreads / 2 - 1)) >> 4;
    float2 g[8][2 * H];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < 2 * H; ++h) g[i][h] = make_float2(0.f, 0.f);
    if (B::STAGES == 2) load(0);
    for (int32_t i = 0; i < n; ++i) {
        load(i + B::STAGES - 1);
        landed<B::STAGES>();
        const float *q = walked(i), *dout = q + B::TILE;
        float p[4][4], ds[4][4];
        weights<D>(p, ds, q, dout, sm, sm + B::TILE, stats(i), a, key0, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sm[B::OFF_P + (ty * 4 + r) * B::PITCH_P + tx + 16 * c] = p[r][c];
                sm[B::OFF_DS + (ty * 4 + r) * B::PITCH_P + tx + 16 * c] = ds[r][c];
            }
        __syncthreads();
        accumulate_t<kBwdRows, H, D + 4>(g, sm + (keys ? B::OFF_DS : B::OFF_P), B::PITCH_P, keys ? q : dout, gy, tx);
        __syncthreads();
    }
    const float scale = keys ? a.scale : 1.f;
    float* out = static_cast<float*>(keys ? a.dk : a.dv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int32_t j = key0 + gy * 8 + i;
        if (j >= end) continue;
        float* y = out + ((int64_t)(t.seq0 + j) * a.Hk + hk) * D + 4 * tx;
#pragma unroll
        for (int h = 0; h < H; ++h)
            store4(y + 64 * h, make_float4(g[i][2 * h].x * scale, g[i][2 * h].y * scale, g[i][2 * h + 1].x * scale,
                                           g[i][2 * h + 1].y * scale));
    }
}

// dq of a tile of rows, over the keys they see.
template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_bwd_q_kernel(AttnArgs a, AttnShape sh)
{
    using B = Bwd<D>;
    constexpr int H = D / 64;
    extern __shared__ __align__(16) float sm[];
    __shared__ AttnTile s_tile;
    __shared__ int s_found;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    wait_for_previous();
    const int32_t unit = blockIdx.x % sh.units, item = blockIdx.x / sh.units;
    const bool bad = a.N > kAttnOrdered && attn_bad(a);
    if (tid < 32) {
        AttnTile t;
        const bool found = attn_find(a, bad, item, sh.tokens, kKeyShift, t);
        if (tid == 0) {
            s_tile = t;
            s_found = found;
        }
    }
    __syncthreads();
    if (!s_found) return;
    const AttnTile t = s_tile;
    const int32_t hk = unit / sh.parts, end = attn_keys(a, t), n = (end + kKeys - 1) >> kKeyShift;
    const RowMap rows(sh, unit, t.row0, t.tokens);
    load_rows<kBwdRows, D>(sm, static_cast<const float*>(a.q), a.q_stride, rows);
    load_rows<kBwdRows, D>(sm + B::TILE, static_cast<const float*>(a.dout), (int64_t)a.Hq * D, rows);
    load_stats(sm + B::OFF_L, a, rows, t.pos0, end);
    auto walked = [&](int32_t i) { return sm + B::OFF_WALK + i % B::STAGES * 2 * B::TILE; };
    auto load = [&](int32_t i) {
        if (i < n) {
            load_keys<D, D + 4>(walked(i), a, static_cast<const float*>(a.k), a.k_stride, t, hk, i * kKeys, end);
            load_keys<D, D + 4>(walked(i) + B::TILE, a, static_cast<const float*>(a.v), a.v_stride, t, hk, i * kKeys,
                                end);
        }
        cp_async_commit();
    };
    float2 dq[4][2 * H];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2 * H; ++h) dq[i][h] = make_float2(0.f, 0.f);
    if (B::STAGES == 2) load(0);
    for (int32_t i = 0; i < n; ++i) {
        load(i + B::STAGES - 1);
        landed<B::STAGES>();
        float p[4][4], ds[4][4];
        weights<D>(p, ds, sm, sm + B::TILE, walked(i), walked(i) + B::TILE, sm + B::OFF_L, a, i * kKeys, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) sm[B::OFF_DS + (ty * 4 + r) * B::PITCH_P + tx + 16 * c] = ds[r][c];
        __syncthreads();
        accumulate<4, H, D + 4>(dq, sm + B::OFF_DS, B::PITCH_P, walked(i), ty, tx);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int32_t token, head;
        if (!rows.at(ty * 4 + i, token, head)) continue;
        float* y = static_cast<float*>(a.dq) + ((int64_t)token * a.Hq + head) * D + 4 * tx;
#pragma unroll
        for (int h = 0; h < H; ++h)
            store4(y + 64 * h, make_float4(dq[i][2 * h].x * a.scale, dq[i][2 * h].y * a.scale,
                                           dq[i][2 * h + 1].x * a.scale, dq[i][2 * h + 1].y * a.scale));
    }
}

// ---------------------------------------------------------------- launch
template <int D, int R> cudaError_t forward_rows(const AttnArgs& a, cudaStream_t stream)
{
    const AttnShape sh = attn_shape(16 * R, a.Hq, a.Hk);
    const int64_t ctas = attn_items(a.N, a.T, sh.tokens) * sh.units * a.splits;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    auto kern = attn_fwd_kernel<D, R>;
    static std::atomic<uint64_t> set{0};
    const cudaError_t e = allow_smem(kern, Fwd<D, R>::SMEM, &set);
    if (e != cudaSuccess) return e;
    return launch_after(kern, launch_config(ctas, kThreads, Fwd<D, R>::SMEM), stream, a, sh);
}
// Rows a thread, by the rows that a group has in a sequence of average length; the largest
// tiles, which read the keys least often, where there are tiles for three quarters of the SMs:
// pieces (attn_splits) then fill the GPU.  With 128 tiles for 152 SMs, tiles of 128 and of 64 rows:
// 1024 tokens, 16 heads of 64 channels 95 and 105 us, in groups of 4 87 and 105; 2048 tokens, 8
// heads of 128 channels 240 and 269; but 512 tokens, 32 heads of 128 channels in groups of 4 92 and
// 79.  With fewer tiles: 4 prompts of 1 to 300 tokens over up to 1000 cached 40 and 33.
int rows_per_thread(int32_t N, int32_t T, int32_t Hq, int32_t Hk)
{
    const int64_t rows = ((int64_t)T + N - 1) / N * (Hq / Hk);
    if (rows > 64) {
        const AttnShape sh = attn_shape(128, Hq, Hk);
        return attn_tiles(N, T, sh.tokens) * sh.units * 4 >= (int64_t)sm_count() * 3 ? 8 : 4;
    }
    return rows > 32 ? 4 : rows > 16 ? 2 : 1;
}

template <int D> cudaError_t forward(const AttnArgs& a, cudaStream_t stream)
{
    switch (rows_per_thread(a.N, a.T, a.Hq, a.Hk)) {
        case 1: return forward_rows<D, 1>(a, stream);
        case 2: return forward_rows<D, 2>(a, stream);
        case 4: return forward_rows<D, 4>(a, stream);
        default: return forward_rows<D, 8>(a, stream);
    }
}

template <typename T, int D> cudaError_t delta(const AttnArgs& a, cudaStream_t stream)
{
    const int64_t rows = (int64_t)a.T * a.Hq, per = Delta<T, D>::PER_BLOCK;
    return launch_after(attn_delta_kernel<T, D>, launch_config((rows + per - 1) / per, 256), stream, a);
}

template <int D> cudaError_t backward(const AttnArgs& a, cudaStream_t stream)
{
    const AttnShape sh = attn_shape(kBwdRows, a.Hq, a.Hk);
    cudaError_t e;
    static std::atomic<uint64_t> set_kv{0}, set_q{0};
    e = allow_smem(attn_bwd_kv_kernel<D>, Bwd<D>::SMEM, &set_kv);
    if (e == cudaSuccess) e = allow_smem(attn_bwd_q_kernel<D>, Bwd<D>::SMEM, &set_q);
    if (e != cudaSuccess) return e;
    e = launch_after(attn_bwd_kv_kernel<D>,
                     launch_config(attn_items(a.N, a.T, kKeys) * a.Hk, kThreads, Bwd<D>::SMEM), stream, a, sh);
    if (e != cudaSuccess) return e;
    return launch_after(attn_bwd_q_kernel<D>,
                        launch_config(attn_items(a.N, a.T, sh.tokens) * sh.units, kThreads, Bwd<D>::SMEM), stream, a,
                        sh);
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs& a, cudaStream_t stream)
{
    const cudaLaunchConfig_t cfg = launch_config(((int64_t)a.T * a.Hq + 7) / 8, 256);
    if (a.bf16)
        return a.D == 64 ? launch_after(attn_join_kernel<__nv_bfloat16, 64>, cfg, stream, a)
                         : launch_after(attn_join_kernel<__nv_bfloat16, 128>, cfg, stream, a);
    return a.D == 64 ? launch_after(attn_join_kernel<float, 64>, cfg, stream, a)
                     : launch_after(attn_join_kernel<float, 128>, cfg, stream, a);
}

// Pieces of two key tiles at least: as many as fill the GPU once on the tensor cores (64 requests
// behind 16384 tokens: 94 us, 110 if twice); three times in FP32, where a tile takes long enough that
// the longest of a causal call would be waited for.  16 heads of 64 channels, twice, three and four times:
// 768 tokens 76, 60 and 58 us, 1024 83, 95 and 93, 1280 160, 119 and 125, 1536 191, 164 and 163, 2048
// 245, 245 and 251; 3000 tokens, 8 heads of 128 channels 613, 482 and 464; 4 prompts of 1 to 300 tokens
// over up to 1000 35.0, 32.7 and 33.8.
int32_t attn_splits(bool bf16, int32_t N, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t kv_most)
{
    if (N == 0 || T == 0) return 1;
    const AttnShape sh = attn_shape(bf16 ? kTcRows : 16 * rows_per_thread(N, T, Hq, Hk), Hq, Hk);
    const int64_t ctas = attn_tiles(N, T, bf16 ? 2 * sh.tokens : sh.tokens) * sh.units;
    const int64_t by_keys = kv_most / (2 * (bf16 ? kTcKeys : kKeys));
    const int64_t by_ctas = (int64_t)sm_count() * (bf16 ? 1 : 3) / ctas;
    const int64_t s = by_ctas < by_keys ? by_ctas : by_keys;
    return (int32_t)(s < 1 ? 1 : s > 64 ? 64 : s);
}

cudaError_t launch_attention(const AttnArgs& a, cudaStream_t stream)
{
    if (a.bf16) return launch_attention_tc(a, stream);
    return a.D == 64 ? forward<64>(a, stream) : forward<128>(a, stream);
}

int64_t attention_bwd_workspace_bytes(int32_t N, int32_t T, int32_t Hq, int32_t Hk, int32_t D)
{
    return ((int64_t)T * Hq * 4 + 255) / 256 * 256 + 16;
}

cudaError_t launch_attention_bwd(const AttnArgs& args, cudaStream_t stream)
{
    AttnArgs a = args;
    a.delta = static_cast<float*>(a.workspace);
    const cudaError_t e =
        a.bf16 ? a.D == 64 ? delta<__nv_bfloat16, 64>(a, stream) : delta<__nv_bfloat16, 128>(a, stream)
        : a.D == 64 ? delta<float, 64>(a, stream) : delta<float, 128>(a, stream);
    if (e != cudaSuccess) return e;
    if (a.bf16) return launch_attention_bwd_tc(a, stream);
    return a.D == 64 ? backward<64>(a, stream) : backward<128>(a, stream);
}

}  // namespace kda
