// kda_qk_norm_rope, kda_qk_norm_rope_append, kda_qk_norm_rope_bwd.
//
// Forward, per row x of D channels (one token, one head):
//     n = x / sqrt(mean x^2 + eps) * w,   (a, b) -> (a cos - b sin, a sin + b cos)
// which is inv * (x_j C_j + x_p S_j) with p the other channel of j's pair, and
// C_j = w_j cos, S_j = -/+ w_p sin the same for all heads of a token.
// Backward, with d = R^T dy (the transposed rotation), n = x rstd, h = d w:
//     dx = rstd (h - n mean(h n)),   dw = sum d n
//
// HBM-bound: a row is read once and written once (backward: x and dy read, dx
// written), 16 bytes a lane.  A row takes D * sizeof(x) / 16 lanes (8, 16 or 32),
// so a warp holds 1, 2 or 4 rows.  Each warp works alone: it takes one token,
// computes that token's cosines and sines once (two angles a lane, exchanged
// through 512 bytes of its own shared memory), keeps its lanes' C and S in
// registers, and runs over the token's heads with kRows rows in flight and the
// next kRows requested before these are worked on; the first are requested before
// the angles.  With few tokens a token's heads are dealt to several warps
// ("slices"), each of which recomputes the angles: that costs less than leaving
// SMs idle.  At 23 bytes per clock and SM a warp has about 170 issue slots per
// step of 512 bytes in and out, so the arithmetic is in pairs (f32x2) and the
// partner channels are exchanged as loaded, before they are unpacked.
//
// Angles: position * inv_freq can be 10^6 radians, where FP32 has lost 0.06.
// The frequency is turned into turns per position as a 64-bit binary fraction
// (an integer product with 1 / (2 pi) in 128 bits; FP64 arithmetic would be
// thirty times slower on this chip); times the position, modulo 2^64, that is the
// fraction of a turn, whose top 32 bits go to sincospif: no argument reduction.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int NT = 256;
constexpr int NW = NT / 32;
constexpr int kMaxPairs = 64;          // rot_dim / 2
constexpr int kRows = 2;               // rows per warp step and lane

template <typename T, int D> struct Layout {
    static constexpr int VEC = 16 / (int)sizeof(T);
    static constexpr int LPR = D / VEC;        // lanes per row
    static constexpr int RPW = 32 / LPR;       // rows per warp
};

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

// 16 bytes as pairs of FP32 values.
template <int N> __device__ __forceinline__ void unpack2(uint4 u, float2 (&f)[N])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (N == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
        f[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        f[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    }
}

template <int N> __device__ __forceinline__ void store2(float* p, const float2 (&f)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 2)
        *reinterpret_cast<float4*>(p + 2 * i) = make_float4(f[i].x, f[i].y, f[i + 1].x, f[i + 1].y);
}
template <int N> __device__ __forceinline__ void store2(__nv_bfloat16* p, const float2 (&f)[N])
{
    if constexpr (N == 4)
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y),
                                                  pack_bf16(f[2].x, f[2].y), pack_bf16(f[3].x, f[3].y));
    else
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y));
}

template <typename T> __device__ __forceinline__ uint4 load16(const T* p)
{
    return *reinterpret_cast<const uint4*>(p);
}

template <int LPR> __device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// The values of the other channels of this lane's pairs, from what its lanes loaded.
template <bool kInter, int N>
__device__ __forceinline__ void partners(uint4 u, const float2 (&f)[N], int lane, float2 (&o)[N])
{
    if constexpr (kInter) {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = make_float2(f[i].y, f[i].x);
    } else {
        uint4 v;
        v.x = __shfl_sync(0xffffffffu, u.x, lane);
        v.y = __shfl_sync(0xffffffffu, u.y, lane);
        v.z = __shfl_sync(0xffffffffu, u.z, lane);
        v.w = __shfl_sync(0xffffffffu, u.w, lane);
        unpack2<N>(v, o);
    }
}

// ---------------------------------------------------------------- angles
// 1 / (2 pi) as a binary fraction of 128 bits.
constexpr uint64_t kTurnHi = 0x28be60db9391054aull, kTurnLo = 0x7f09d5f47d4d3770ull;

// inv_freq (radians per position) as turns per position modulo one, in units of
// 2^-64: its 24-bit significand times 1 / (2 pi), shifted by its exponent.
__device__ __forceinline__ uint64_t turns_of(float inv_freq)
{
    const uint32_t bits = __float_as_uint(inv_freq);
    const int e = (bits >> 23) & 255;
    const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int s = 150 - (e ? e : 1);               // inv_freq = m 2^-s
    const uint64_t p0 = m * kTurnLo, c = __umul64hi(m, kTurnLo);
    const uint64_t p1 = m * kTurnHi + c;
    const uint64_t p2 = __umul64hi(m, kTurnHi) + (p1 < c);
    // (p2 p1 p0) / 2^128 2^-s turns: bits from 2^-1 to 2^-64
    uint64_t t;
    if (s >= 64)
        t = s >= 128 ? 0 : p2 >> (s - 64);
    else if (s > 0)
        t = (p1 >> s) | (p2 << (64 - s));
    else
        t = s == 0 ? p1 : s > -64 ? (p1 << -s) | (p0 >> (64 + s)) : 0;
    return bits >> 31 ? 0 - t : t;
}

// The lane's two frequencies (pairs lane and lane + 32).
__device__ __forceinline__ void lane_turns(const RopeArgs& a, int lane, uint64_t (&f)[2])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int p = lane + 32 * i;
        f[i] = p < a.rot / 2 ? turns_of(a.inv_freq[p]) : 0;
    }
}

// Cosines and sines of the warp's token into its table.
__device__ __forceinline__ void warp_angles(const RopeArgs& a, const uint64_t (&f)[2],
                                            float2* table, int32_t pos, int lane)
{
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int p = lane + 32 * i;
        if (p < a.rot / 2) {
            const uint64_t turn = f[i] * (uint64_t)(int64_t)pos;
            // [-2^31, 2^31) of 2^-32 turns each; sincospif takes half turns
            const float half = (float)(int32_t)(uint32_t)(turn >> 32) * 0x1p-31f;
            float sn, cs;
            sincospif(half, &sn, &cs);
            table[p] = make_float2(cs * a.rope_scale, sn * a.rope_scale);
        }
    }
    __syncwarp();
}

// Channel ch's cosine and signed sine (1 and 0 where it is not rotated), and the
// other channel of its pair.
__device__ __forceinline__ float2 channel_turn(const RopeArgs& a, const float2* table, bool inter,
                                               int ch, int* other)
{
    *other = ch;
    if (ch >= a.rot) return make_float2(1.f, 0.f);
    const int h = a.rot >> 1;
    const bool second = inter ? (ch & 1) : ch >= h;
    *other = inter ? ch ^ 1 : second ? ch - h : ch + h;
    const float2 t = table[inter ? ch >> 1 : second ? ch - h : ch];
    return make_float2(t.x, second ? t.y : -t.y);
}

// The lane that holds the other channels of this lane's pairs (half layout).
__device__ __forceinline__ int partner_lane(const RopeArgs& a, int lane, int chan, int vec)
{
    if (chan >= a.rot) return lane;
    const int d = a.rot / 2 / vec;
    return chan < a.rot / 2 ? lane + d : lane - d;
}

// The weights of both kinds in shared memory (ones where there are none).
template <int D> __device__ __forceinline__ void block_weights(const RopeArgs& a, float (*w)[D])
{
    for (int i = threadIdx.x; i < 2 * D; i += NT) {
        const float* p = i < D ? a.q_weight : a.k_weight;
        w[i / D][i % D] = a.norm && p != nullptr ? p[i % D] : 1.f;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- forward
// items = T * slices; warp-item i: token i / slices, rows of slice i % slices of
// the q heads, then of the k heads, then (append) of the v heads.
template <typename TIn, typename TOut, int D, bool kAppend, bool kInter>
__global__ void __launch_bounds__(NT, 3) qk_rope_kernel(RopeArgs a, int slices)
{
    using L = Layout<TIn, D>;
    constexpr int NP = L::VEC / 2;                         // pairs of values per lane
    __shared__ float2 table[NW][kMaxPairs];
    __shared__ float weights[2][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / L::LPR, chan = (lane % L::LPR) * L::VEC;
    const int partner = partner_lane(a, lane, chan, L::VEC);
    const int64_t items = (int64_t)a.T * slices, nwarps = (int64_t)gridDim.x * NW;
    const int step = slices * L::RPW;
    constexpr int kKinds = kAppend ? 3 : 2;
    uint64_t f[2];
    bool ready = false;
    for (int64_t i = (int64_t)blockIdx.x * NW + warp;; i += nwarps) {
        // every warp of the block passes here once before its first item
        const bool any = i < items;
        const int64_t t = any ? (int64_t)((uint32_t)i / (uint32_t)slices) : 0;
        const int top = any ? (int)(i - t * slices) * L::RPW : INT32_MAX;   // uniform in the warp
        const int32_t pos = any ? a.positions[t] : 0;
        int64_t slot = 0;
        if (kAppend && any) slot = a.slots[t];
        const bool stored = !kAppend || (slot >= 0 && slot < a.num_slots);
        const int kinds = stored ? kKinds : 1;
        const TIn* src[kKinds];
        src[0] = static_cast<const TIn*>(a.q) + t * a.q_stride;
        src[1] = static_cast<const TIn*>(a.k) + t * a.k_stride;
        if constexpr (kAppend) src[2] = static_cast<const TIn*>(a.v) + t * a.v_stride;
        // the step's place: rows top + row, top + row + step, ... of kind `kind`
        int kind = 0, row = 0;
        auto settle = [&] {
            // the heads first: a slot is not waited for before q's rows are requested
            while (top + row >= (kind == 0 ? a.Hq : a.Hk) && kind < kinds) {
                ++kind;
                row = 0;
            }
        };
        auto request = [&](uint4 (&u)[kRows]) {
            if (kind > 0 && kind >= kinds) return;
            const TIn* x = kind == 0 ? src[0] : kind == 1 ? src[1] : src[kKinds - 1];
            const int H = kind == 0 ? a.Hq : a.Hk;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int h = top + sub + row + r * step;
                u[r] = make_uint4(0, 0, 0, 0);
                if (h < H) u[r] = load16(x + (int64_t)h * D + chan);
            }
        };
        uint4 next[kRows];
        if (any) {
            settle();
            request(next);
        }
        if (!ready) {
            lane_turns(a, lane, f);
            block_weights<D>(a, weights);
            ready = true;
        }
        if (!any) break;
        if (kAppend && slot >= a.num_slots && lane == 0) report_status(a.status, KDA_ERR_DEVICE_ARG);
        warp_angles(a, f, table[warp], pos, lane);
        int64_t paged = 0;                                 // the slot's row of head 0
        if (kAppend && stored) {
            const int64_t page = slot / a.page;
            paged = (page * a.Hk * a.page + (slot - page * a.page)) * D;
        }

        float2 c[NP], s[NP];
        int have = -1;                                     // the kind that c and s are for
        while (kind < kinds) {
            uint4 u[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) u[r] = next[r];
            const int now = kind, at = row;
            row += kRows * step;
            settle();
            request(next);
            if (now != have && now < 2) {
                have = now;
#pragma unroll
                for (int j = 0; j < L::VEC; ++j) {
                    int o;
                    const float2 cs = channel_turn(a, table[warp], kInter, chan + j, &o);
                    const float x = cs.x * weights[now][chan + j], y = cs.y * weights[now][o];
                    if (j & 1) { c[j / 2].y = x; s[j / 2].y = y; }
                    else { c[j / 2].x = x; s[j / 2].x = y; }
                }
            }
            TOut* y;
            int64_t hstep = D;
            if (now == 0) {
                y = static_cast<TOut*>(a.q_out) + t * a.Hq * D;
            } else if (!kAppend) {
                y = static_cast<TOut*>(a.k_out) + t * a.Hk * D;
            } else {
                y = static_cast<TOut*>(now == 1 ? a.k_out : a.v_out) + paged;
                hstep = (int64_t)a.page * D;
            }
            const int H = now == 0 ? a.Hq : a.Hk;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (top + at + r * step >= H) break;       // warp-uniform
                const int h = top + sub + at + r * step;
                float2 x[NP];
                unpack2<NP>(u[r], x);
                if (!kAppend || now < 2) {
                    float2 o[NP];
                    partners<kInter, NP>(u[r], x, partner, o);
                    float inv = 1.f;
                    if (a.norm) {
                        float2 ss = mul2(x[0], x[0]);
#pragma unroll
                        for (int j = 1; j < NP; ++j) ss = fma2(x[j], x[j], ss);
                        inv = rsqrtf(row_sum<L::LPR>(ss.x + ss.y) * (1.f / D) + a.eps);
                    }
#pragma unroll
                    for (int j = 0; j < NP; ++j)
                        x[j] = mul2(fma2(o[j], s[j], mul2(x[j], c[j])), both(inv));
                }
                if (h < H) store2<NP>(y + h * hstep + chan, x);
            }
        }
    }
}

// ---------------------------------------------------------------- backward
// Rows of one kind of one token.
template <typename TIn, typename TDy, typename TOut, int D, bool kInter>
__device__ __forceinline__ void grad_rows(const RopeArgs& a, const TIn* x, const TDy* dy, TOut* dx,
                                          int H, int top, int sub, int step, int chan, int partner,
                                          const float* weights,
                                          const float2 (&c)[Layout<TIn, D>::VEC / 2],
                                          const float2 (&s)[Layout<TIn, D>::VEC / 2],
                                          float2 (&dw)[Layout<TIn, D>::VEC / 2])
{
    using L = Layout<TIn, D>;
    constexpr int VEC = L::VEC, NP = VEC / 2;
    // 16-byte loads of dy per lane (8 bytes of one where dy is BF16 and x FP32)
    constexpr int ND = VEC * (int)sizeof(TDy) >= 16 ? VEC * (int)sizeof(TDy) / 16 : 1;
    constexpr int PV = 8 / (int)sizeof(TDy);               // pairs in 16 bytes of dy
    float2 w[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) w[j] = make_float2(weights[chan + 2 * j], weights[chan + 2 * j + 1]);
    auto request = [&](int at, uint4 (&u)[kRows], uint4 (&g)[kRows][ND]) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int h = top + sub + at + r * step;
            u[r] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < ND; ++i) g[r][i] = make_uint4(0, 0, 0, 0);
            if (h < H) {
                u[r] = load16(x + (int64_t)h * D + chan);
                const TDy* p = dy + (int64_t)h * D + chan;
                if constexpr (VEC * sizeof(TDy) == 8) {
                    const uint2 v = *reinterpret_cast<const uint2*>(p);
                    g[r][0].x = v.x;
                    g[r][0].y = v.y;
                } else {
#pragma unroll
                    for (int i = 0; i < ND; ++i) g[r][i] = load16(p + i * (16 / (int)sizeof(TDy)));
                }
            }
        }
    };
    uint4 un[kRows], gn[kRows][ND];
    request(0, un, gn);
    for (int at = 0; top + at < H; at += kRows * step) {
        uint4 u[kRows], g[kRows][ND];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            u[r] = un[r];
#pragma unroll
            for (int i = 0; i < ND; ++i) g[r][i] = gn[r][i];
        }
        request(at + kRows * step, un, gn);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (top + at + r * step >= H) break;           // warp-uniform
            const int h = top + sub + at + r * step;
            float2 f[NP], d[NP], o[NP];
            unpack2<NP>(u[r], f);
#pragma unroll
            for (int i = 0; i < ND; ++i) {
                float2 part[PV], other[PV];
                unpack2<PV>(g[r][i], part);
                partners<kInter, PV>(g[r][i], part, partner, other);
#pragma unroll
                for (int j = 0; j < PV; ++j)
                    if (i * PV + j < NP) {
                        d[i * PV + j] = part[j];
                        o[i * PV + j] = other[j];
                    }
            }
            // the transposed rotation: s carries its signs
#pragma unroll
            for (int j = 0; j < NP; ++j) d[j] = fma2(o[j], s[j], mul2(d[j], c[j]));
            if (a.norm) {
                float2 ss = mul2(f[0], f[0]), hx = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 1; j < NP; ++j) ss = fma2(f[j], f[j], ss);
                float2 hw[NP];
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    hw[j] = mul2(d[j], w[j]);
                    hx = fma2(hw[j], f[j], hx);
                }
                const float rstd = rsqrtf(row_sum<L::LPR>(ss.x + ss.y) * (1.f / D) + a.eps);
                // n mean(h n) = x rstd^2 mean(h x)
                const float m = row_sum<L::LPR>(hx.x + hx.y) * (1.f / D) * rstd * rstd;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    dw[j] = fma2(mul2(f[j], both(rstd)), d[j], dw[j]);
                    d[j] = mul2(fma2(f[j], both(-m), hw[j]), both(rstd));
                }
            }
            if (h < H) store2<NP>(dx + (int64_t)h * D + chan, d);
        }
    }
}

// Sum of the CTA's dw over its warps and row groups, in a fixed order.
template <int NP, int LPR, int D>
__device__ __forceinline__ void block_dw(const float2 (&dw)[NP], float (*red)[D], float* out)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        float2 x = dw[j];
#pragma unroll
        for (int m = 16; m >= LPR; m >>= 1) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, m);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, m);
        }
        if (lane < LPR) *reinterpret_cast<float2*>(&red[warp][2 * (lane * NP + j)]) = x;
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < D; ch += NT) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) x += red[w][ch];
        out[ch] = x;
    }
}

template <typename TIn, typename TDy, typename TOut, int D, bool kInter>
__global__ void __launch_bounds__(NT, 2) qk_rope_bwd_kernel(RopeArgs a, int slices)
{
    using L = Layout<TIn, D>;
    constexpr int NP = L::VEC / 2;
    __shared__ float2 table[NW][kMaxPairs];
    __shared__ float weights[2][D];
    __shared__ float red[NW][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / L::LPR, chan = (lane % L::LPR) * L::VEC;
    const int partner = partner_lane(a, lane, chan, L::VEC);
    uint64_t f[2];
    lane_turns(a, lane, f);
    block_weights<D>(a, weights);
    const int64_t items = (int64_t)a.T * slices, nwarps = (int64_t)gridDim.x * NW;
    const int step = slices * L::RPW;
    let_next_start();
    float2 dwq[NP], dwk[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) dwq[j] = dwk[j] = make_float2(0.f, 0.f);
    for (int64_t i = (int64_t)blockIdx.x * NW + warp; i < items; i += nwarps) {
        const int64_t t = (uint32_t)i / (uint32_t)slices;
        const int top = (int)(i - t * slices) * L::RPW;
        warp_angles(a, f, table[warp], a.positions[t], lane);
        float2 c[NP], s[NP];
#pragma unroll
        for (int j = 0; j < L::VEC; ++j) {
            int o;
            const float2 cs = channel_turn(a, table[warp], kInter, chan + j, &o);
            if (j & 1) { c[j / 2].y = cs.x; s[j / 2].y = -cs.y; }
            else { c[j / 2].x = cs.x; s[j / 2].x = -cs.y; }
        }
        grad_rows<TIn, TDy, TOut, D, kInter>(
            a, static_cast<const TIn*>(a.q) + t * a.q_stride,
            static_cast<const TDy*>(a.dq) + t * a.Hq * D, static_cast<TOut*>(a.q_out) + t * a.Hq * D,
            a.Hq, top, sub, step, chan, partner, weights[0], c, s, dwq);
        grad_rows<TIn, TDy, TOut, D, kInter>(
            a, static_cast<const TIn*>(a.k) + t * a.k_stride,
            static_cast<const TDy*>(a.dk) + t * a.Hk * D, static_cast<TOut*>(a.k_out) + t * a.Hk * D,
            a.Hk, top, sub, step, chan, partner, weights[1], c, s, dwk);
    }
    if (a.norm && (a.q_wgrad != nullptr || a.k_wgrad != nullptr)) {
        float* out = a.partials + (int64_t)blockIdx.x * 2 * D;
        block_dw<NP, L::LPR, D>(dwq, red, out);
        block_dw<NP, L::LPR, D>(dwk, red, out + D);
    }
}

// Adds up the CTAs' weight gradients: 32 channels a block, 32 partial sums each.
__global__ void __launch_bounds__(1024) dw_sum_kernel(const float* partials, int ctas, int D,
                                                      float* q_wgrad, float* k_wgrad)
{
    __shared__ float red[32][33];
    const int col = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int ch = blockIdx.x * 32 + col;
    float x = 0.f;
    wait_for_previous();
    for (int i = part; i < ctas; i += 32) x += partials[(int64_t)i * 2 * D + ch];
    red[part][col] = x;
    __syncthreads();
    if (part == 0) {
        x = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) x += red[i][col];
        float* out = ch < D ? q_wgrad : k_wgrad;
        if (out != nullptr) out[ch < D ? ch : ch - D] = x;
    }
}

constexpr int kFwdCtasPerSm = 3, kBwdCtasPerSm = 2;    // resident, by registers
int64_t bwd_ctas_bound() { return (int64_t)sm_count() * kBwdCtasPerSm; }

// Warps per token.  `steps` warp steps of rows make a token; a warp-item costs its
// share of them and a start (the angles, C and S) of about kStart steps, and items
// run in rounds of `warps`.  The count with the shortest schedule: one where the
// tokens alone fill many rounds, as many as the rows allow for a few tokens.
constexpr int kStart = 4;
int slices_for(int64_t T, int steps, int64_t warps)
{
    int best = 1;
    int64_t least = INT64_MAX;
    for (int s = 1; s <= steps && s <= 64; ++s) {
        if (T * s > INT32_MAX) break;
        const int64_t rounds = (T * s + warps - 1) / warps;
        const int64_t cost = rounds * ((steps + s - 1) / s + kStart);
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}
int row_steps(int H, int rpw) { return (H + rpw - 1) / rpw; }

template <typename TIn, typename TOut, int D, bool kInter>
cudaError_t launch_fwd(const RopeArgs& a, bool append, cudaStream_t stream)
{
    const int64_t resident = (int64_t)sm_count() * kFwdCtasPerSm;
    constexpr int rpw = Layout<TIn, D>::RPW;
    const int slices = slices_for(a.T, row_steps(a.Hq, rpw), resident * NW);
    int64_t blocks = ((int64_t)a.T * slices + NW - 1) / NW;
    // beyond eight rounds of CTAs each warp takes more tokens instead
    if (blocks > 8 * resident) blocks = 8 * resident;
    if (append)
        qk_rope_kernel<TIn, TOut, D, true, kInter><<<(unsigned)blocks, NT, 0, stream>>>(a, slices);
    else
        qk_rope_kernel<TIn, TOut, D, false, kInter><<<(unsigned)blocks, NT, 0, stream>>>(a, slices);
    return cudaGetLastError();
}

template <typename TIn, typename TOut>
cudaError_t launch_fwd_d(const RopeArgs& a, bool append, cudaStream_t stream)
{
    if (a.interleaved)
        return a.D == 64 ? launch_fwd<TIn, TOut, 64, true>(a, append, stream)
                         : launch_fwd<TIn, TOut, 128, true>(a, append, stream);
    return a.D == 64 ? launch_fwd<TIn, TOut, 64, false>(a, append, stream)
                     : launch_fwd<TIn, TOut, 128, false>(a, append, stream);
}

template <typename TIn, typename TDy, typename TOut, int D>
cudaError_t launch_bwd(const RopeArgs& a, cudaStream_t stream)
{
    // every CTA leaves a partial sum, so there are no more than are resident
    const int64_t resident = bwd_ctas_bound();
    const int slices = slices_for(a.T, row_steps(a.Hq, Layout<TIn, D>::RPW), resident * NW);
    int64_t blocks = ((int64_t)a.T * slices + NW - 1) / NW;
    if (blocks > resident) blocks = resident;
    if (a.interleaved)
        qk_rope_bwd_kernel<TIn, TDy, TOut, D, true><<<(unsigned)blocks, NT, 0, stream>>>(a, slices);
    else
        qk_rope_bwd_kernel<TIn, TDy, TOut, D, false><<<(unsigned)blocks, NT, 0, stream>>>(a, slices);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.norm && (a.q_wgrad != nullptr || a.k_wgrad != nullptr)) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * D / 32);
        cfg.blockDim = dim3(1024);
        e = launch_after(dw_sum_kernel, cfg, stream, a.partials, (int)blocks, D, a.q_wgrad, a.k_wgrad);
    }
    return e;
}

template <typename TIn, typename TDy>
cudaError_t launch_bwd_o(const RopeArgs& a, cudaStream_t stream)
{
    if (a.D == 64)
        return a.out_bf16 ? launch_bwd<TIn, TDy, __nv_bfloat16, 64>(a, stream)
                          : launch_bwd<TIn, TDy, float, 64>(a, stream);
    return a.out_bf16 ? launch_bwd<TIn, TDy, __nv_bfloat16, 128>(a, stream)
                      : launch_bwd<TIn, TDy, float, 128>(a, stream);
}

}  // namespace

int64_t qk_rope_bwd_workspace_bytes(int32_t D) { return bwd_ctas_bound() * 2 * D * 4; }

cudaError_t launch_qk_rope(const RopeArgs& a, bool append, cudaStream_t stream)
{
    if (a.x_bf16)
        return a.out_bf16 ? launch_fwd_d<__nv_bfloat16, __nv_bfloat16>(a, append, stream)
                          : launch_fwd_d<__nv_bfloat16, float>(a, append, stream);
    return a.out_bf16 ? launch_fwd_d<float, __nv_bfloat16>(a, append, stream)
                      : launch_fwd_d<float, float>(a, append, stream);
}

cudaError_t launch_qk_rope_bwd(const RopeArgs& a, cudaStream_t stream)
{
    if (a.x_bf16)
        return a.dy_bf16 ? launch_bwd_o<__nv_bfloat16, __nv_bfloat16>(a, stream)
                         : launch_bwd_o<__nv_bfloat16, float>(a, stream);
    return a.dy_bf16 ? launch_bwd_o<float, __nv_bfloat16>(a, stream)
                     : launch_bwd_o<float, float>(a, stream);
}

}  // namespace kda
