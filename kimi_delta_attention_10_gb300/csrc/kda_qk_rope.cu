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
// registers, and runs over the token's heads.  Rows come through a ring of four
// asynchronous copies per warp (the first are under way before the angles are
// computed): 32 warps keep 48 KB of an SM in flight without a register, and the
// partner channels of the half layout are one more read of the ring instead of four
// shuffles.  At 23 bytes per clock and SM a warp has about 170 issue slots per step
// of 512 bytes in and out, so the arithmetic is in pairs (f32x2).  With few tokens a
// token's heads are dealt to several warps ("slices"), each of which recomputes the
// angles: that costs less than leaving SMs idle.
//
// Measured (us, and the share of the rate of a plain copy): append of 30392 BF16 tokens of
// 64 + 8 heads of 128 channels 196.5 (93%; 83% of the issue slots), forward of 2048 FP32 tokens
// of 64 + 64 heads 43.8 (90%), backward of 16384 BF16 tokens of 64 + 8 heads 146 (91%), 64 or
// 129 tokens 4.5.  Few heads and many tokens spend their issue slots on the angles: 16384 BF16
// tokens of 5 + 1 heads 25.8 (29%; 61% of the issue slots).
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
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int NT = 256;
constexpr int NW = NT / 32;
constexpr int kMaxPairs = 64;          // rot_dim / 2

template <typename T, int D> struct Layout {
    static constexpr int VEC = 16 / (int)sizeof(T);
    static constexpr int LPR = D / VEC;        // lanes per row
    static constexpr int RPW = 32 / LPR;       // rows per warp
};

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

// One instruction, where a product of two 64-bit factors is half a dozen.
__device__ __forceinline__ int64_t wide(int a, int b) { return (int64_t)a * b; }

template <int LPR> __device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

__device__ __forceinline__ uint4 lds16(const unsigned char* p) { return *reinterpret_cast<const uint4*>(p); }

// The values of the other channels of this lane's pairs: its own, swapped, or the
// partner lane's, at `other` in the ring.
template <bool kInter, int N>
__device__ __forceinline__ void partners(const float2 (&f)[N], const unsigned char* other, float2 (&o)[N])
{
    if constexpr (kInter) {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = make_float2(f[i].y, f[i].x);
    } else {
        unpack2<N>(lds16(other), o);
    }
}

template <int N> __device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async8(void* dst, const void* src, bool valid)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(tc::smem_u32(dst)), "l"(src),
                 "r"(valid ? 8 : 0)
                 : "memory");
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

// Cosines and signed sines of the lane's VEC channels (1 and 0 where they are not
// rotated), in pairs of channels, and the first of the other channels of their pairs.
// rot_dim is a multiple of 16, so that a lane's channels are all rotated or none, and in
// the half layout all first or all second ones: their pairs lie side by side in the table.
template <int VEC, bool kInter>
__device__ __forceinline__ int lane_turn(const RopeArgs& a, const float2* table, int chan,
                                         float2 (&c)[VEC / 2], float2 (&s)[VEC / 2])
{
    if (chan >= a.rot) {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            c[j] = make_float2(1.f, 1.f);
            s[j] = make_float2(-0.f, -0.f);               // a zero keeps its sign too
        }
        return chan;
    }
    if constexpr (kInter) {
        // (cos, sin) of pair chan / 2 + j
#pragma unroll
        for (int j = 0; j < VEC / 2; j += 2) {
            const float4 t = *reinterpret_cast<const float4*>(table + chan / 2 + j);
            c[j] = make_float2(t.x, t.x);
            s[j] = make_float2(-t.y, t.y);
            c[j + 1] = make_float2(t.z, t.z);
            s[j + 1] = make_float2(-t.w, t.w);
        }
        return chan;
    } else {
        const int h = a.rot >> 1;
        const bool second = chan >= h;
        const float sign = second ? 1.f : -1.f;
        const float2* at = table + (second ? chan - h : chan);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const float4 t = *reinterpret_cast<const float4*>(at + 2 * j);
            c[j] = make_float2(t.x, t.z);
            s[j] = make_float2(t.y * sign, t.w * sign);
        }
        return second ? chan - h : chan + h;
    }
}

// x c + o s.  A channel that is not rotated takes nothing of another, which may be infinite:
// in the half layout its o is zero.
template <bool kInter>
__device__ __forceinline__ float2 turn(float2 x, float2 o, float2 c, float2 s, bool turned)
{
    float2 y = mul2(x, c);
    if (!kInter || turned) y = fma2(o, s, y);
    return y;
}

// N pairs of consecutive weights.
template <int N> __device__ __forceinline__ void weight_pairs(const float* w, float2 (&f)[N])
{
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const float4 t = *reinterpret_cast<const float4*>(w + 2 * j);
        f[j] = make_float2(t.x, t.y);
        f[j + 1] = make_float2(t.z, t.w);
    }
}

// The lane that holds the other channels of this lane's pairs (half layout).
__device__ __forceinline__ int partner_lane(const RopeArgs& a, int lane, int chan, int vec)
{
    if (chan >= a.rot) return lane;
    const int d = a.rot / 2 / vec;
    return chan < a.rot / 2 ? lane + d : lane - d;
}

// What all tokens share, in shared memory: the weights of both kinds (ones where there are
// none) and the frequencies.
template <int D> struct Common {
    float weights[2][D];
    uint64_t turns[kMaxPairs];

    __device__ __forceinline__ void load(const RopeArgs& a)
    {
        for (int i = threadIdx.x; i < 2 * D; i += NT) {
            const float* p = i < D ? a.q_weight : a.k_weight;
            weights[i / D][i % D] = a.norm && p != nullptr ? p[i % D] : 1.f;
        }
        // the last warps: the first ones may have most of the weights
        const int i = NT - 1 - (int)threadIdx.x;
        if (i < a.rot / 2) turns[i] = turns_of(a.inv_freq[i]);
        __syncthreads();
    }
    // The lane's two frequencies: pairs lane and lane + 32.
    __device__ __forceinline__ void lane_turns(const RopeArgs& a, int lane, uint64_t (&f)[2]) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) f[i] = lane + 32 * i < a.rot / 2 ? turns[lane + 32 * i] : 0;
    }
};

// ---------------------------------------------------------------- forward
constexpr int kRing = 4;

// items = T * slices; warp-item i: token i / slices, rows of slice i % slices of
// the q heads, then of the k heads, then (append) of the v heads.
template <typename TIn, typename TOut, int D, bool kAppend, bool kInter>
__global__ void __launch_bounds__(NT, 4) qk_rope_kernel(RopeArgs a, int log_slices)
{
    using L = Layout<TIn, D>;
    constexpr int NP = L::VEC / 2;                         // pairs of values per lane
    constexpr int kKinds = kAppend ? 3 : 2;
    __shared__ __align__(16) float2 table[NW][kMaxPairs];
    __shared__ __align__(16) Common<D> common;
    __shared__ __align__(16) unsigned char ring[NW][kRing][kInter ? 512 : 528];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / L::LPR, chan = (lane % L::LPR) * L::VEC;
    const bool turned = chan < a.rot;
    // where in a slot of the ring the other channels of the lane's pairs lie; zeros for none
    const int partner = turned ? partner_lane(a, lane, chan, L::VEC) * 16 : 512;
    if (!kInter && lane < kRing)
        *reinterpret_cast<uint4*>(&ring[warp][lane][512]) = make_uint4(0, 0, 0, 0);
    const int64_t items = (int64_t)a.T << log_slices;
    const int nwarps = gridDim.x * NW;
    const int step = L::RPW << log_slices;
    wait_for_previous();
    uint64_t f[2];
    bool ready = false;
    for (int64_t i = (int64_t)blockIdx.x * NW + warp;; i += nwarps) {
        // every warp of the block passes here once before its first item
        const bool any = i < items;
        const int t = any ? (int)(i >> log_slices) : 0;
        const int top = ((int)i & ((1 << log_slices) - 1)) * L::RPW;    // uniform in the warp
        const int32_t pos = any ? a.positions[t] : 0;
        int64_t slot = 0;
        if (kAppend && any) slot = a.slots[t];
        const int lane_off = (top + sub) * D + chan;
        const TIn* src[3] = {static_cast<const TIn*>(a.q) + wide(t, a.q_stride) + lane_off,
                             static_cast<const TIn*>(a.k) + wide(t, a.k_stride) + lane_off,
                             kAppend ? static_cast<const TIn*>(a.v) + wide(t, a.v_stride) + lane_off : nullptr};
        // the next copy: rows row .. of kind `want`
        int want = 0, row = top;
        const TIn* p = src[0];
        auto settle = [&] {
            if (want == 0 && row >= a.Hq) {
                want = 1;
                row = top;
                p = src[1];
            }
            if (want == 1 && row >= a.Hk) {
                want = 2;
                row = top;
                p = src[2];
            }
            if (want == 2 && (!kAppend || row >= a.Hk)) want = 3;
        };
        int put = 0;                                       // ring slot of the next copy
        auto request = [&] {
            if (want < 3) {
                const bool valid = row + sub < (want == 0 ? a.Hq : a.Hk);
                tc::cp_async16(&ring[warp][put][lane * 16], valid ? p : static_cast<const TIn*>(a.q), valid);
                p += step * D;
                row += step;
                settle();
            }
            tc::cp_async_commit();
            put = (put + 1) % kRing;
        };
        if (any) {
            settle();
#pragma unroll
            for (int k = 0; k < kRing - 1; ++k) request();
        }
        if (!ready) {
            common.load(a);
            common.lane_turns(a, lane, f);
            ready = true;
        }
        if (!any) break;
        warp_angles(a, f, table[warp], pos, lane);
        const bool stored = !kAppend || (slot >= 0 && slot < a.num_slots);
        if (kAppend && slot >= a.num_slots && lane == 0) report_status(a.status, KDA_ERR_DEVICE_ARG);
        int64_t paged = 0;                                 // the slot's row of head 0
        if (kAppend && stored) {
            const int64_t page = slot >> 32 ? slot / a.page : (uint32_t)slot / (uint32_t)a.page;
            paged = (page * a.Hk * a.page + (slot - page * a.page)) * D;
        }
        int get = 0;
#pragma unroll
        for (int kind = 0; kind < kKinds; ++kind) {
            const int H = kind == 0 ? a.Hq : a.Hk;
            if (top >= H) continue;
            const int64_t hstep = kAppend && kind > 0 ? (int64_t)a.page * D : D;
            TOut* y = (kind == 0   ? static_cast<TOut*>(a.q_out) + wide(t, a.Hq * D)
                       : !kAppend  ? static_cast<TOut*>(a.k_out) + wide(t, a.Hk * D)
                       : kind == 1 ? static_cast<TOut*>(a.k_out) + paged
                                   : static_cast<TOut*>(a.v_out) + paged) +
                      (top + sub) * hstep + chan;
            const int64_t jump = step * hstep;
            float2 c[NP], s[NP];
            if (kind < 2) {
                const int o = lane_turn<L::VEC, kInter>(a, table[warp], chan, c, s);
                if (a.norm) {
                    float2 w[NP], v[NP];
                    weight_pairs<NP>(&common.weights[kind][chan], w);
                    weight_pairs<NP>(&common.weights[kind][o], v);
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        c[j] = mul2(c[j], w[j]);
                        // neighbours' weights trade places with them
                        s[j] = mul2(s[j], kInter ? make_float2(v[j].y, v[j].x) : v[j]);
                    }
                }
            }
            for (int h = top; h < H; h += step, y += jump) {
                copies_wait<kRing - 2>();
                __syncwarp();                              // all lanes' parts; the last step's are read
                const unsigned char* at = ring[warp][get];
                float2 x[NP];
                unpack2<NP>(lds16(at + lane * 16), x);
                if (kind < 2) {
                    float2 o[NP];
                    partners<kInter, NP>(x, at + partner, o);
                    request();
                    float inv = 1.f;
                    if (a.norm) {
                        float2 ss = mul2(x[0], x[0]);
#pragma unroll
                        for (int j = 1; j < NP; ++j) ss = fma2(x[j], x[j], ss);
                        inv = rsqrtf(row_sum<L::LPR>(ss.x + ss.y) * (1.f / D) + a.eps);
                    }
#pragma unroll
                    for (int j = 0; j < NP; ++j)
                        x[j] = mul2(turn<kInter>(x[j], o[j], c[j], s[j], turned), both(inv));
                } else {
                    request();
                }
                get = (get + 1) % kRing;
                if (h + sub < H && (kind == 0 || stored)) store2<NP>(y, x);
            }
        }
        copies_wait<0>();
        __syncwarp();
    }
}

// ---------------------------------------------------------------- backward
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

// A warp's ring of x and dy rows, in the half layout with zeros at each slot's end; DYB: bytes
// of dy a lane takes (8, 16 or 32).
template <typename TIn, typename TDy, int D, bool kInter> struct BwdRing {
    static constexpr int DYB = Layout<TIn, D>::VEC * (int)sizeof(TDy);
    static constexpr int SLOTS = DYB == 32 ? 3 : 4;
    static constexpr int ZEROS = 512 + 32 * DYB, BYTES = ZEROS + (kInter ? 0 : DYB == 32 ? 32 : 16);
};

template <typename TIn, typename TDy, typename TOut, int D, bool kInter>
__global__ void __launch_bounds__(NT, 2) qk_rope_bwd_kernel(RopeArgs a, int log_slices)
{
    using L = Layout<TIn, D>;
    using R = BwdRing<TIn, TDy, D, kInter>;
    constexpr int NP = L::VEC / 2, DYB = R::DYB, S = R::SLOTS;
    __shared__ __align__(16) float2 table[NW][kMaxPairs];
    __shared__ __align__(16) Common<D> common;
    __shared__ __align__(16) unsigned char ring[NW][S][R::BYTES];
    static_assert(sizeof(ring) >= NW * D * sizeof(float), "the sums of dw reuse the ring");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / L::LPR, chan = (lane % L::LPR) * L::VEC;
    const bool turned = chan < a.rot;
    const int partner = turned ? 512 + partner_lane(a, lane, chan, L::VEC) * DYB : R::ZEROS;
    if (!kInter && lane < S)
        for (int i = R::ZEROS; i < R::BYTES; i += 16)
            *reinterpret_cast<uint4*>(&ring[warp][lane][i]) = make_uint4(0, 0, 0, 0);
    const int64_t items = (int64_t)a.T << log_slices;
    const int nwarps = gridDim.x * NW;
    const int step = L::RPW << log_slices;
    wait_for_previous();
    uint64_t f[2];
    bool ready = false;
    float2 dwq[NP], dwk[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) dwq[j] = dwk[j] = make_float2(0.f, 0.f);
    for (int64_t i = (int64_t)blockIdx.x * NW + warp;; i += nwarps) {
        const bool any = i < items;
        const int t = any ? (int)(i >> log_slices) : 0;
        const int top = ((int)i & ((1 << log_slices) - 1)) * L::RPW;
        const int32_t pos = any ? a.positions[t] : 0;
        const int lane_off = (top + sub) * D + chan;
        const TIn* xq = static_cast<const TIn*>(a.q) + wide(t, a.q_stride) + lane_off;
        const TIn* xk = static_cast<const TIn*>(a.k) + wide(t, a.k_stride) + lane_off;
        const TDy* yq = static_cast<const TDy*>(a.dq) + wide(t, a.Hq * D) + lane_off;
        const TDy* yk = static_cast<const TDy*>(a.dk) + wide(t, a.Hk * D) + lane_off;
        int want = 0, row = top;
        const TIn* px = xq;
        const TDy* py = yq;
        auto settle = [&] {
            if (want == 0 && row >= a.Hq) {
                want = 1;
                row = top;
                px = xk;
                py = yk;
            }
            if (want == 1 && row >= a.Hk) want = 2;
        };
        int put = 0;
        auto request = [&] {
            if (want < 2) {
                const bool valid = row + sub < (want == 0 ? a.Hq : a.Hk);
                unsigned char* at = ring[warp][put];
                tc::cp_async16(at + lane * 16, valid ? px : static_cast<const TIn*>(a.q), valid);
                const TDy* from = valid ? py : static_cast<const TDy*>(a.dq);
                if constexpr (DYB == 8) {
                    cp_async8(at + 512 + lane * 8, from, valid);
                } else {
#pragma unroll
                    for (int k = 0; k < DYB / 16; ++k)
                        tc::cp_async16(at + 512 + lane * DYB + 16 * k, from + k * (16 / (int)sizeof(TDy)),
                                       valid);
                }
                px += step * D;
                py += step * D;
                row += step;
                settle();
            }
            tc::cp_async_commit();
            put = (put + 1) % S;
        };
        if (any) {
            settle();
#pragma unroll
            for (int k = 0; k < S - 1; ++k) request();
        }
        if (!ready) {
            common.load(a);
            common.lane_turns(a, lane, f);
            ready = true;
        }
        if (!any) break;
        warp_angles(a, f, table[warp], pos, lane);
        float2 c[NP], s[NP];                               // of the transposed rotation
        lane_turn<L::VEC, kInter>(a, table[warp], chan, c, s);
#pragma unroll
        for (int j = 0; j < NP; ++j)
            if (turned) s[j] = make_float2(-s[j].x, -s[j].y);
        int get = 0;
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const int H = kind == 0 ? a.Hq : a.Hk;
            if (top >= H) continue;
            TOut* dx = static_cast<TOut*>(kind == 0 ? a.q_out : a.k_out) + wide(t, H * D) + lane_off;
            float2 w[NP];
            weight_pairs<NP>(&common.weights[kind][chan], w);
            for (int h = top; h < H; h += step, dx += step * D) {
                copies_wait<S - 2>();
                __syncwarp();
                const unsigned char* at = ring[warp][get];
                float2 x[NP], d[NP], o[NP];
                unpack2<NP>(lds16(at + lane * 16), x);
                if constexpr (DYB == 8) {
                    // four BF16 values
                    const uint2 u = *reinterpret_cast<const uint2*>(at + 512 + lane * 8);
                    float2 v[4];
                    unpack2<4>(make_uint4(u.x, u.y, 0, 0), v);
                    d[0] = v[0];
                    d[1] = v[1];
                    if constexpr (kInter) {
                        o[0] = make_float2(d[0].y, d[0].x);
                        o[1] = make_float2(d[1].y, d[1].x);
                    } else {
                        const uint2 z = *reinterpret_cast<const uint2*>(at + partner);
                        unpack2<4>(make_uint4(z.x, z.y, 0, 0), v);
                        o[0] = v[0];
                        o[1] = v[1];
                    }
                } else {
                    constexpr int PV = 8 / (int)sizeof(TDy);   // pairs in 16 bytes of dy
#pragma unroll
                    for (int k = 0; k < DYB / 16; ++k) {
                        float2 v[PV], z[PV];
                        unpack2<PV>(lds16(at + 512 + lane * DYB + 16 * k), v);
                        partners<kInter, PV>(v, at + partner + 16 * k, z);
#pragma unroll
                        for (int j = 0; j < PV; ++j) {
                            d[k * PV + j] = v[j];
                            o[k * PV + j] = z[j];
                        }
                    }
                }
                request();
                get = (get + 1) % S;
#pragma unroll
                for (int j = 0; j < NP; ++j) d[j] = turn<kInter>(d[j], o[j], c[j], s[j], turned);
                if (a.norm) {
                    float2 ss = mul2(x[0], x[0]), hx = make_float2(0.f, 0.f);
#pragma unroll
                    for (int j = 1; j < NP; ++j) ss = fma2(x[j], x[j], ss);
                    float2 hw[NP];
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        hw[j] = mul2(d[j], w[j]);
                        hx = fma2(hw[j], x[j], hx);
                    }
                    // rows past the heads are zeros, which an infinite factor would make NaN in dw
                    const float ms = row_sum<L::LPR>(ss.x + ss.y) * (1.f / D) + a.eps;
                    const float rstd = h + sub < H ? rsqrtf(ms) : 0.f;
                    // n mean(h n) = x rstd^2 mean(h x)
                    const float m = row_sum<L::LPR>(hx.x + hx.y) * (1.f / D) * rstd * rstd;
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        float2& dw = kind == 0 ? dwq[j] : dwk[j];
                        dw = fma2(mul2(x[j], both(rstd)), d[j], dw);
                        d[j] = mul2(fma2(x[j], both(-m), hw[j]), both(rstd));
                    }
                }
                if (h + sub < H) store2<NP>(dx, d);
            }
        }
        copies_wait<0>();
        __syncwarp();
    }
    if (a.norm && (a.q_wgrad != nullptr || a.k_wgrad != nullptr)) {
        float* out = a.partials + (int64_t)blockIdx.x * 2 * D;
        float (*red)[D] = reinterpret_cast<float (*)[D]>(&ring[0][0][0]);
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

constexpr int kFwdCtasPerSm = 4, kBwdCtasPerSm = 2;    // resident, by registers
int64_t bwd_ctas_bound() { return (int64_t)sm_count() * kBwdCtasPerSm; }

// log2 of the warps per token (a power of two: a shift tells an item's token).  With s
// slices an item costs its share of the token's row steps and a start (the angles, C and
// S), measured at about three steps where the arithmetic is near the issue limit (BF16)
// and one where it hides behind memory (FP32).  Items run `warps` at a time: the whole
// takes T s / warps items' time (but no less than 0.45 of one, where too few warps are
// left to fill the memory's latency) and a quarter of an item at the end.  Measured with 64 + 8 heads of 128 channels (us): 16384 BF16 tokens 100,
// 108, 131 for 1, 2, 4 slices; 129 tokens 14.2, 5.8, 5.9 for 1, 8, 16; 16384 FP32 tokens
// 191, 181, 178 for 1, 2, 4.
int slices_for(int64_t T, int q_steps, int k_steps, int k_kinds, float start, int64_t warps)
{
    float least = 0.f;
    const int most = q_steps > k_steps ? q_steps : k_steps;
    int best = 0;
    for (int log = 0; log <= 6 && (1 << log) < 2 * most && (T << log) <= INT32_MAX; ++log) {
        const int s = 1 << log, steps = (q_steps + s - 1) / s + k_kinds * ((k_steps + s - 1) / s);
        const float fill = (float)(T * s) / (float)warps;
        const float cost = ((fill > 0.45f ? fill : 0.45f) + 0.25f) * (steps + start);
        if (log == 0 || cost < least) {
            least = cost;
            best = log;
        }
    }
    return best;
}
int row_steps(int H, int rpw) { return (H + rpw - 1) / rpw; }
template <typename T> constexpr float start_steps() { return sizeof(T) == 2 ? 3.f : 1.f; }

template <typename TIn, typename TOut, int D, bool kInter>
cudaError_t launch_fwd(const RopeArgs& a, bool append, cudaStream_t stream)
{
    const int64_t resident = (int64_t)sm_count() * kFwdCtasPerSm;
    constexpr int rpw = Layout<TIn, D>::RPW;
    const int log_slices = slices_for(a.T, row_steps(a.Hq, rpw), row_steps(a.Hk, rpw), append ? 2 : 1,
                                  start_steps<TIn>(), resident * NW);
    int64_t blocks = (((int64_t)a.T << log_slices) + NW - 1) / NW;
    // beyond eight rounds of CTAs each warp takes more tokens instead
    if (blocks > 8 * resident) blocks = 8 * resident;
    return launch_after(append ? qk_rope_kernel<TIn, TOut, D, true, kInter>
                               : qk_rope_kernel<TIn, TOut, D, false, kInter>,
                        launch_config(blocks, NT), stream, a, log_slices);
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
    constexpr int rpw = Layout<TIn, D>::RPW;
    const int log_slices = slices_for(a.T, row_steps(a.Hq, rpw), row_steps(a.Hk, rpw), 1,
                                  sizeof(TIn) == 2 ? 3.f : 2.5f,
                                  resident * NW);
    int64_t blocks = (((int64_t)a.T << log_slices) + NW - 1) / NW;
    if (blocks > resident) blocks = resident;
    cudaError_t e = launch_after(a.interleaved ? qk_rope_bwd_kernel<TIn, TDy, TOut, D, true>
                                               : qk_rope_bwd_kernel<TIn, TDy, TOut, D, false>,
                                 launch_config(blocks, NT), stream, a, log_slices);
    if (e == cudaSuccess && a.norm && (a.q_wgrad != nullptr || a.k_wgrad != nullptr)) {
        e = launch_after(dw_sum_kernel, launch_config(2 * D / 32, 1024), stream, a.partials, (int)blocks,
                         D, a.q_wgrad, a.k_wgrad);
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
