// kda_qk_norm_rope, kda_qk_norm_rope_append, kda_qk_norm_rope_bwd.
//
// Forward, per row x of D channels (one token, one head):
//     n = x / sqrt(mean x^2 + eps) * w,   (a, b) -> (a cos - b sin, a sin + b cos)
// Backward, with d = R^T dy (the transposed rotation), n = x rstd, h = d w:
//     dx = rstd (h - n mean(h n)),   dw = sum d n
//
// HBM-bound: a row is read once and written once (backward: x and dy read, dx
// written), 16 bytes a lane.  A row takes D * sizeof(x) / 16 lanes (8, 16 or 32),
// so a warp holds 1, 2 or 4 rows.  Each warp works alone: it takes one token,
// computes that token's cosines and sines once (two angles a lane, exchanged
// through 512 bytes of its own shared memory), keeps the ones its lanes need in
// registers, and runs over the token's heads with kRows rows in flight.  With
// few tokens a token's heads are dealt to several warps ("slices"), each of which
// recomputes the angles: that costs less than leaving SMs idle.
//
// Angles: position * inv_freq can be 10^6 radians, where FP32 has lost 0.06.
// The frequency is turned once per warp into turns per position as a 64-bit
// binary fraction; times the position, modulo 2^64, that is the exact fraction
// of a turn, whose top 32 bits go to sincospif: no argument reduction at all,
// two integer multiplies an angle.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int NT = 256;
constexpr int NW = NT / 32;
constexpr int kMaxPairs = 64;          // rot_dim / 2
constexpr int kRows = 4;               // row loads in flight per lane

template <typename T, int D> struct Layout {
    static constexpr int VEC = 16 / (int)sizeof(T);
    static constexpr int LPR = D / VEC;        // lanes per row
    static constexpr int RPW = 32 / LPR;       // rows per warp
};

// inv_freq (radians per position) as turns per position, a binary fraction of
// 64 bits modulo one turn.
__device__ __forceinline__ uint64_t turns_of(float inv_freq)
{
    double x = (double)inv_freq * 0.15915494309189533577;   // 1 / (2 pi)
    x -= floor(x);
    // x < 1 has 53 bits: the product is exact, and at most 2^64 - 2^11
    return __double2ull_rz(x * 18446744073709551616.0);
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

// Cosines and sines of the warp's token, for the lane's channels: value j of the
// lane's vector becomes c[j] * own + s[j] * partner.
template <int VEC>
__device__ __forceinline__ void lane_rotation(const RopeArgs& a, const uint64_t (&f)[2],
                                              float2* table, int32_t pos, int lane, int chan,
                                              float (&c)[VEC], float (&s)[VEC])
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
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int ch = chan + j;
        c[j] = 1.f;
        s[j] = 0.f;
        if (ch < a.rot) {
            const int h = a.rot / 2;
            const bool second = a.interleaved ? (ch & 1) : ch >= h;
            const float2 t = table[a.interleaved ? ch >> 1 : second ? ch - h : ch];
            c[j] = t.x;
            s[j] = second ? t.y : -t.y;
        }
    }
}

// The lane that holds the other channels of this lane's pairs (half layout).
__device__ __forceinline__ int partner_lane(const RopeArgs& a, int lane, int chan, int vec)
{
    if (a.interleaved || chan >= a.rot) return lane;
    const int d = a.rot / 2 / vec;
    return chan < a.rot / 2 ? lane + d : lane - d;
}

template <int VEC>
__device__ __forceinline__ void rotate(float (&x)[VEC], const float (&c)[VEC],
                                       const float (&s)[VEC], bool interleaved, int partner)
{
    float o[VEC];
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = x[j ^ 1];
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = __shfl_sync(0xffffffffu, x[j], partner);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = fmaf(x[j], c[j], o[j] * s[j]);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

template <int VEC>
__device__ __forceinline__ void lane_weight(const float* w, bool norm, int chan, float (&r)[VEC])
{
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[j] = norm && w != nullptr ? w[chan + j] : 1.f;
}

template <typename T>
__device__ __forceinline__ uint4 load16(const T* p)
{
    return *reinterpret_cast<const uint4*>(p);
}

// Where row h of the warp's token goes: dense, or a page.
struct Dense {
    int64_t base, step;
    __device__ __forceinline__ int64_t at(int h) const { return base + h * step; }
};

// One token's rows of one kind (q or k): rows first, first + step, ... < H.
template <typename TIn, typename TOut, int D>
__device__ __forceinline__ void norm_rope_rows(const RopeArgs& a, const TIn* x, TOut* y, Dense to,
                                               int H, int first, int step, int chan, int partner,
                                               const float* weight,
                                               const float (&c)[Layout<TIn, D>::VEC],
                                               const float (&s)[Layout<TIn, D>::VEC])
{
    using L = Layout<TIn, D>;
    constexpr int VEC = L::VEC;
    float w[VEC];
    lane_weight<VEC>(weight, a.norm, chan, w);
    const int top = first - first % L::RPW;                 // the warp's first row: uniform
    for (int h0 = 0; top + h0 < H; h0 += kRows * step) {
        uint4 u[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int h = first + h0 + r * step;
            u[r] = h < H ? load16(x + (int64_t)h * D + chan) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (top + h0 + r * step >= H) break;            // warp-uniform
            const int h = first + h0 + r * step;
            float f[VEC];
            Vec16<TIn>::unpack(u[r], f);
            if (a.norm) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < VEC; ++j) ss = fmaf(f[j], f[j], ss);
                const float inv = 1.f / sqrtf(row_sum<L::LPR>(ss) * (1.f / D) + a.eps);
#pragma unroll
                for (int j = 0; j < VEC; ++j) f[j] *= inv * w[j];
            }
            rotate<VEC>(f, c, s, a.interleaved, partner);
            if (h < H && y != nullptr) store_vec<VEC>(y + to.at(h) + chan, f);
        }
    }
}

// One token's value rows, copied to their page.
template <typename TIn, typename TOut, int D>
__device__ __forceinline__ void copy_rows(const TIn* x, TOut* y, Dense to, int H, int first,
                                          int step, int chan)
{
    constexpr int VEC = Layout<TIn, D>::VEC;
    for (int h0 = first; h0 < H; h0 += kRows * step) {
        uint4 u[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (h0 + r * step < H) u[r] = load16(x + (int64_t)(h0 + r * step) * D + chan);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int h = h0 + r * step;
            if (h < H) {
                float f[VEC];
                Vec16<TIn>::unpack(u[r], f);
                store_vec<VEC>(y + to.at(h) + chan, f);
            }
        }
    }
}

// items = T * slices; warp-item i: token i / slices, rows of slice i % slices.
template <typename TIn, typename TOut, int D, bool kAppend>
__global__ void __launch_bounds__(NT) qk_rope_kernel(RopeArgs a, int slices)
{
    using L = Layout<TIn, D>;
    __shared__ float2 table[NW][kMaxPairs];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / L::LPR, chan = (lane % L::LPR) * L::VEC;
    const int partner = partner_lane(a, lane, chan, L::VEC);
    uint64_t f[2];
    lane_turns(a, lane, f);
    const int64_t items = (int64_t)a.T * slices;
    const int64_t nwarps = (int64_t)gridDim.x * NW;
    const int step = slices * L::RPW;
    for (int64_t i = (int64_t)blockIdx.x * NW + warp; i < items; i += nwarps) {
        const int64_t t = i / slices;
        const int first = (int)(i - t * slices) * L::RPW + sub;
        float c[L::VEC], s[L::VEC];
        lane_rotation<L::VEC>(a, f, table[warp], a.positions[t], lane, chan, c, s);
        norm_rope_rows<TIn, TOut, D>(a, static_cast<const TIn*>(a.q) + t * a.q_stride,
                                     static_cast<TOut*>(a.q_out), Dense{t * a.Hq * D, D}, a.Hq,
                                     first, step, chan, partner, a.q_weight, c, s);
        const TIn* k = static_cast<const TIn*>(a.k) + t * a.k_stride;
        if (!kAppend) {
            norm_rope_rows<TIn, TOut, D>(a, k, static_cast<TOut*>(a.k_out),
                                         Dense{t * a.Hk * D, D}, a.Hk, first, step, chan, partner,
                                         a.k_weight, c, s);
        } else {
            const int64_t slot = a.slots[t];
            if (slot < 0 || slot >= a.num_slots) {
                if (slot >= 0 && lane == 0) report_status(a.status, KDA_ERR_DEVICE_ARG);
                continue;
            }
            const int64_t page = slot / a.page;
            const Dense to{(page * a.Hk * a.page + (slot - page * a.page)) * D,
                           (int64_t)a.page * D};
            norm_rope_rows<TIn, TOut, D>(a, k, static_cast<TOut*>(a.k_out), to, a.Hk, first, step,
                                         chan, partner, a.k_weight, c, s);
            copy_rows<TIn, TOut, D>(static_cast<const TIn*>(a.v) + t * a.v_stride,
                                    static_cast<TOut*>(a.v_out), to, a.Hk, first, step, chan);
        }
    }
}

// ---------------------------------------------------------------- backward
template <typename TIn, typename TDy, typename TOut, int D>
__device__ __forceinline__ void grad_rows(const RopeArgs& a, const TIn* x, const TDy* dy, TOut* dx,
                                          int H, int first, int step, int chan, int partner,
                                          const float* weight,
                                          const float (&c)[Layout<TIn, D>::VEC],
                                          const float (&s)[Layout<TIn, D>::VEC],
                                          float (&dw)[Layout<TIn, D>::VEC])
{
    using L = Layout<TIn, D>;
    constexpr int VEC = L::VEC;
    constexpr int R = 2;                   // rows in flight: two loads each
    // 16-byte loads of dy per lane: VEC values
    constexpr int ND = VEC * (int)sizeof(TDy) >= 16 ? VEC * (int)sizeof(TDy) / 16 : 1;
    float w[VEC];
    lane_weight<VEC>(weight, a.norm, chan, w);
    const int top = first - first % L::RPW;
    for (int h0 = 0; top + h0 < H; h0 += R * step) {
        uint4 u[R], g[R][ND];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int h = first + h0 + r * step;
            u[r] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < ND; ++i) g[r][i] = make_uint4(0, 0, 0, 0);
            if (h < H) {
                u[r] = load16(x + (int64_t)h * D + chan);
                const TDy* p = dy + (int64_t)h * D + chan;
                if constexpr (VEC * sizeof(TDy) == 8) {
                    const uint2 half = *reinterpret_cast<const uint2*>(p);
                    g[r][0].x = half.x;
                    g[r][0].y = half.y;
                } else {
#pragma unroll
                    for (int i = 0; i < ND; ++i)
                        g[r][i] = load16(p + i * (16 / (int)sizeof(TDy)));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (top + h0 + r * step >= H) break;            // warp-uniform
            const int h = first + h0 + r * step;
            float f[VEC], d[VEC];
            Vec16<TIn>::unpack(u[r], f);
#pragma unroll
            for (int i = 0; i < ND; ++i) {
                float part[16 / sizeof(TDy)];
                Vec16<TDy>::unpack(g[r][i], part);
#pragma unroll
                for (int j = 0; j < (int)(16 / sizeof(TDy)); ++j)
                    if (i * (int)(16 / sizeof(TDy)) + j < VEC)
                        d[i * (int)(16 / sizeof(TDy)) + j] = part[j];
            }
            rotate<VEC>(d, c, s, a.interleaved, partner);   // s holds the transposed signs
            if (a.norm) {
                float ss = 0.f, hx = 0.f;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    ss = fmaf(f[j], f[j], ss);
                    hx = fmaf(d[j] * w[j], f[j], hx);
                }
                ss = row_sum<L::LPR>(ss);
                hx = row_sum<L::LPR>(hx);
                const float rstd = 1.f / sqrtf(ss * (1.f / D) + a.eps);
                const float m = hx * rstd * (1.f / D);      // mean(h n)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float n = f[j] * rstd;
                    dw[j] = fmaf(d[j], n, dw[j]);
                    d[j] = rstd * (d[j] * w[j] - n * m);
                }
            }
            if (h < H) store_vec<VEC>(dx + (int64_t)h * D + chan, d);
        }
    }
}

// Sum of the CTA's dw over its warps and row groups, in a fixed order.
template <int VEC, int LPR, int D>
__device__ __forceinline__ void block_dw(const float (&dw)[VEC], float (*red)[D], float* out)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        float x = dw[j];
#pragma unroll
        for (int m = 16; m >= LPR; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
        if (lane < LPR) red[warp][lane * VEC + j] = x;
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < D; ch += NT) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) x += red[w][ch];
        out[ch] = x;
    }
}

template <typename TIn, typename TDy, typename TOut, int D>
__global__ void __launch_bounds__(NT) qk_rope_bwd_kernel(RopeArgs a, int slices)
{
    using L = Layout<TIn, D>;
    __shared__ float2 table[NW][kMaxPairs];
    __shared__ float red[NW][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / L::LPR, chan = (lane % L::LPR) * L::VEC;
    const int partner = partner_lane(a, lane, chan, L::VEC);
    uint64_t f[2];
    lane_turns(a, lane, f);
    const int64_t items = (int64_t)a.T * slices;
    const int64_t nwarps = (int64_t)gridDim.x * NW;
    const int step = slices * L::RPW;
    float dwq[L::VEC], dwk[L::VEC];
#pragma unroll
    for (int j = 0; j < L::VEC; ++j) dwq[j] = dwk[j] = 0.f;
    for (int64_t i = (int64_t)blockIdx.x * NW + warp; i < items; i += nwarps) {
        const int64_t t = i / slices;
        const int first = (int)(i - t * slices) * L::RPW + sub;
        float c[L::VEC], s[L::VEC];
        lane_rotation<L::VEC>(a, f, table[warp], a.positions[t], lane, chan, c, s);
#pragma unroll
        for (int j = 0; j < L::VEC; ++j) s[j] = -s[j];
        grad_rows<TIn, TDy, TOut, D>(a, static_cast<const TIn*>(a.q) + t * a.q_stride,
                                     static_cast<const TDy*>(a.dq) + t * a.Hq * D,
                                     static_cast<TOut*>(a.q_out) + t * a.Hq * D, a.Hq, first, step,
                                     chan, partner, a.q_weight, c, s, dwq);
        grad_rows<TIn, TDy, TOut, D>(a, static_cast<const TIn*>(a.k) + t * a.k_stride,
                                     static_cast<const TDy*>(a.dk) + t * a.Hk * D,
                                     static_cast<TOut*>(a.k_out) + t * a.Hk * D, a.Hk, first, step,
                                     chan, partner, a.k_weight, c, s, dwk);
    }
    if (a.norm && (a.q_wgrad != nullptr || a.k_wgrad != nullptr)) {
        float* out = a.partials + (int64_t)blockIdx.x * 2 * D;
        block_dw<L::VEC, L::LPR, D>(dwq, red, out);
        block_dw<L::VEC, L::LPR, D>(dwk, red, out + D);
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

constexpr int kBwdCtasPerSm = 4;
int64_t bwd_ctas_bound()
{
    const int sms = device_sm_count();
    return (int64_t)(sms > 0 ? sms : 152) * kBwdCtasPerSm;
}

// Warps per token and CTAs of a launch with at most `most` CTAs.
void shape_of(int64_t T, int rows, int rpw, int64_t most, int* slices, unsigned* blocks)
{
    // enough warps for every CTA slot, but at least one full step of rows each
    const int64_t want = (most * NW + T - 1) / T;
    const int64_t can = (rows + rpw - 1) / rpw;
    int64_t s = want < can ? want : can;
    if (s < 1) s = 1;
    int64_t b = (T * s + NW - 1) / NW;
    if (b > most) b = most;
    *slices = (int)s;
    *blocks = (unsigned)b;
}

template <typename TIn, typename TOut, int D>
cudaError_t launch_fwd(const RopeArgs& a, bool append, cudaStream_t stream)
{
    const int sms = device_sm_count();
    int slices;
    unsigned blocks;
    shape_of(a.T, a.Hq, Layout<TIn, D>::RPW, (int64_t)(sms > 0 ? sms : 152) * 4, &slices, &blocks);
    if (append)
        qk_rope_kernel<TIn, TOut, D, true><<<blocks, NT, 0, stream>>>(a, slices);
    else
        qk_rope_kernel<TIn, TOut, D, false><<<blocks, NT, 0, stream>>>(a, slices);
    return cudaGetLastError();
}

template <typename TIn, typename TOut>
cudaError_t launch_fwd_d(const RopeArgs& a, bool append, cudaStream_t stream)
{
    return a.D == 64 ? launch_fwd<TIn, TOut, 64>(a, append, stream)
                     : launch_fwd<TIn, TOut, 128>(a, append, stream);
}

template <typename TIn, typename TDy, typename TOut, int D>
cudaError_t launch_bwd(const RopeArgs& a, cudaStream_t stream)
{
    int slices;
    unsigned blocks;
    shape_of(a.T, a.Hq, Layout<TIn, D>::RPW, bwd_ctas_bound(), &slices, &blocks);
    qk_rope_bwd_kernel<TIn, TDy, TOut, D><<<blocks, NT, 0, stream>>>(a, slices);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.norm && (a.q_wgrad != nullptr || a.k_wgrad != nullptr)) {
        dw_sum_kernel<<<2 * D / 32, 1024, 0, stream>>>(a.partials, (int)blocks, D, a.q_wgrad,
                                                       a.k_wgrad);
        e = cudaGetLastError();
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
