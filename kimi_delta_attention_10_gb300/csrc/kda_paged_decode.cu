// kda_paged_decode for FP32 caches, on CUDA cores (IEEE FP32 products), and the join
// of split rows for either type.
//
//     s_t = scale q . k_t,   out = sum e^(s_t) v_t / sum e^(s_t)
//
// HBM-bound: every k and v is read once, 2 D values a token and key-value head.
// Each warp works alone on batches of eight consecutive tokens (which lie in one
// page): a row takes D / 4 lanes, 16 bytes each, straight from memory to
// registers, keys and values of the batch together in flight; the products with
// the unit's query rows (in registers, scaled by scale * log2 e) are summed over
// the row's lanes by shuffles, and one pass keeps the running maximum m, sum l and
// output o in base 2.  The CTA's warps take different batches of the same row and
// merge (m, l, o) through shared memory at the end of it.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "kda_paged_sched.cuh"

namespace kda {
namespace {

constexpr int NT = 256;
constexpr int NW = NT / 32;
constexpr int kBatch = 8;              // tokens per warp step
constexpr int kTileShift = 6;          // 64 tokens: one batch per warp

template <int D, int GT>
__global__ void __launch_bounds__(NT) paged_decode_kernel(DecodeArgs a, DecodeShape sh, int chunks)
{
    using T = float;
    constexpr int VEC = 4;
    constexpr int LPR = D / VEC, RPW = 32 / LPR;
    constexpr int TB = kBatch / RPW;               // tokens per row group and step
    __shared__ float s_m[NW][GT], s_l[NW][GT];
    __shared__ float s_o[NW][GT][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / LPR, chan = (lane % LPR) * VEC;
    const int G = a.Hq / a.Hk;
    // The warps are dealt to head chunks of GT heads; those of one chunk share the row's tokens.
    const int chunk = warp % chunks, stream = warp / chunks, streams = NW / chunks;
    char* ws = static_cast<char*>(a.workspace);
    float2* ws_ml = reinterpret_cast<float2*>(ws + decode_ml_offset(a.N));
    float* ws_o = reinterpret_cast<float*>(ws + decode_o_offset(a.N, sh));
    let_next_start();
    const DecodeRange rg = decode_range<NT>(a, sh, reinterpret_cast<int64_t*>(ws));
    const T* kc = static_cast<const T*>(a.k);
    const T* vc = static_cast<const T*>(a.v);
    const int groups = sh.units / a.Hk;            // units per key-value head
    const float qscale = a.scale * kLog2e;

    int64_t pos = rg.begin, at = rg.at;
    int32_t n = rg.n;
    while (pos < rg.end) {
        const int32_t L = decode_len(a, n), tiles = tiles_of(L, sh.tile_shift);
        if (pos >= at + (int64_t)tiles * sh.units) {
            at += (int64_t)tiles * sh.units;
            ++n;
            continue;
        }
        const int32_t u = (int32_t)((pos - at) / tiles);
        const int32_t tile0 = (int32_t)(pos - at - (int64_t)u * tiles);
        const int32_t tile1 = (int32_t)min((int64_t)tiles, tile0 + (rg.end - pos));
        const int hk = u / groups;
        const int head0 = (u - hk * groups) * sh.heads + chunk * GT;   // in the group of G
        const int t0 = tile0 << sh.tile_shift, t1 = min(L, tile1 << sh.tile_shift);

        float q[GT][VEC], o[GT][VEC], m[GT], l[GT];
#pragma unroll
        for (int g = 0; g < GT; ++g) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (head0 + g < G)
                x = *reinterpret_cast<const uint4*>(
                    static_cast<const T*>(a.q) +
                    ((int64_t)n * a.Hq + hk * G + head0 + g) * D + chan);
            Vec16<T>::unpack(x, q[g]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                q[g][j] *= qscale;
                o[g][j] = 0.f;
            }
            m[g] = -CUDART_INF_F;
            l[g] = 0.f;
        }
        const int32_t* row = a.table + (int64_t)n * a.max_pages;
        for (int b = t0 + stream * kBatch; b < t1; b += streams * kBatch) {
            const int32_t page = row[b >> a.page_shift];
            if ((uint32_t)page >= (uint32_t)a.num_pages) {
                if (lane == 0) report_status(a.status, KDA_ERR_DEVICE_ARG);
                continue;
            }
            const int64_t base = ((((int64_t)page * a.Hk + hk) << a.page_shift) +
                                  (b & ((1 << a.page_shift) - 1))) * D + chan;
            uint4 ku[TB], vu[TB];
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                const int t = j * RPW + sub;
                ku[j] = vu[j] = make_uint4(0, 0, 0, 0);     // rows past the end: never read
                if (b + t < t1) {
                    ku[j] = __ldg(reinterpret_cast<const uint4*>(kc + base + (int64_t)t * D));
                    vu[j] = __ldg(reinterpret_cast<const uint4*>(vc + base + (int64_t)t * D));
                }
            }
            float s[TB][GT];
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                float kf[VEC];
                Vec16<T>::unpack(ku[j], kf);
                const bool live = b + j * RPW + sub < t1;
#pragma unroll
                for (int g = 0; g < GT; ++g) {
                    float x = 0.f;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) x = fmaf(q[g][i], kf[i], x);
#pragma unroll
                    for (int k = LPR / 2; k > 0; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
                    s[j][g] = live ? x : -CUDART_INF_F;
                }
            }
#pragma unroll
            for (int g = 0; g < GT; ++g) {
                float top = m[g];
#pragma unroll
                for (int j = 0; j < TB; ++j) top = fmaxf(top, s[j][g]);
                // a row group that has seen no token yet: nothing to subtract
                const float ref = top == -CUDART_INF_F ? 0.f : top;
                const float keep = exp2f(m[g] - ref);
                m[g] = top;
                l[g] *= keep;
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[g][i] *= keep;
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    s[j][g] = exp2f(s[j][g] - ref);
                    l[g] += s[j][g];
                }
            }
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                float vf[VEC];
                Vec16<T>::unpack(vu[j], vf);
#pragma unroll
                for (int g = 0; g < GT; ++g)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) o[g][i] = fmaf(s[j][g], vf[i], o[g][i]);
            }
        }
        // merge the warp's row groups, then the chunk's warps
#pragma unroll
        for (int g = 0; g < GT; ++g) {
            float top = m[g];
#pragma unroll
            for (int k = LPR; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
            const float keep = top == -CUDART_INF_F ? 0.f : exp2f(m[g] - top);
            float lg = l[g] * keep;
#pragma unroll
            for (int k = LPR; k < 32; k <<= 1) lg += __shfl_xor_sync(0xffffffffu, lg, k);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float x = o[g][i] * keep;
#pragma unroll
                for (int k = LPR; k < 32; k <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
                if (sub == 0) s_o[warp][g][chan + i] = x;
            }
            if (lane == 0) {
                s_m[warp][g] = top;
                s_l[warp][g] = lg;
            }
        }
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == tiles;
        const int64_t piece = 2 * (int64_t)blockIdx.x + (tile0 == 0 ? 1 : 0);
        for (int i = threadIdx.x; i < chunks * GT * D; i += NT) {
            const int ch = i % D, g = (i / D) % GT, c = i / (D * GT);
            const int head = (u - hk * groups) * sh.heads + c * GT + g;
            if (c * GT + g >= sh.heads || head >= G) continue;
            float top = -CUDART_INF_F;
            for (int w = c; w < NW; w += chunks) top = fmaxf(top, s_m[w][g]);
            float lsum = 0.f, x = 0.f;
            if (top != -CUDART_INF_F)
                for (int w = c; w < NW; w += chunks) {
                    const float keep = exp2f(s_m[w][g] - top);
                    lsum += s_l[w][g] * keep;
                    x += s_o[w][g][ch] * keep;
                }
            if (whole) {
                const int64_t r = (int64_t)n * a.Hq + hk * G + head;
                const float y = x / lsum;
                if (a.out_bf16)
                    store_one(static_cast<__nv_bfloat16*>(a.out) + r * D + ch, y);
                else
                    store_one(static_cast<float*>(a.out) + r * D + ch, y);
                if (ch == 0 && a.lse != nullptr) a.lse[r] = top * kLn2 + logf(lsum);
            } else {
                const int64_t r = piece * sh.heads + c * GT + g;
                ws_o[r * D + ch] = x;
                if (ch == 0) ws_ml[r] = make_float2(top, lsum);
            }
        }
        __syncthreads();
        pos += tile1 - tile0;
    }
}

// One query head of one request per block: nothing to do for a whole row, zeros
// for an empty request, and for a split row the joined pieces in the CTAs' order.
template <int D>
__global__ void __launch_bounds__(NT) decode_join_kernel(DecodeArgs a, DecodeShape sh)
{
    constexpr int P = NT / D;                      // pieces taken side by side
    __shared__ float s_x[P][D], s_l[P];
    const int h = blockIdx.x % a.Hq;
    const int32_t n = blockIdx.x / a.Hq;
    const int G = a.Hq / a.Hk, hk = h / G, groups = sh.units / a.Hk;
    const int g = (h - hk * G) % sh.heads;
    const int u = hk * groups + (h - hk * G) / sh.heads;
    const int ch = threadIdx.x % D, part = threadIdx.x / D;
    const char* ws = static_cast<const char*>(a.workspace);
    const int64_t* prefix = reinterpret_cast<const int64_t*>(ws);
    const float2* ws_ml = reinterpret_cast<const float2*>(ws + decode_ml_offset(a.N));
    const float* ws_o = reinterpret_cast<const float*>(ws + decode_o_offset(a.N, sh));
    wait_for_previous();
    const int64_t p0 = prefix[n], tiles = prefix[n + 1] - p0, W = prefix[a.N] * sh.units;
    const int64_t r = blockIdx.x;
    float y = 0.f, lse = -CUDART_INF_F;
    if (tiles > 0) {
        const int64_t first = p0 * sh.units + u * tiles, last = first + tiles - 1;
        // the CTA of tile x: the last b with b W / B <= x
        const int64_t B = W < sh.ctas ? W : sh.ctas;
        const int64_t b0 = ((first + 1) * B - 1) / W, b1 = ((last + 1) * B - 1) / W;
        if (b0 == b1) return;                      // whole: written by its CTA
        // the row begins in the first CTA's tiles, and before the others'
        float top = -CUDART_INF_F;
        for (int64_t b = b0; b <= b1; ++b)
            top = fmaxf(top, ws_ml[(2 * b + (b == b0)) * sh.heads + g].x);
        float x = 0.f, l = 0.f;
        if (top != -CUDART_INF_F)
            for (int64_t b = b0 + part; b <= b1; b += P) {
                const int64_t i = (2 * b + (b == b0)) * sh.heads + g;
                const float2 ml = ws_ml[i];
                const float keep = exp2f(ml.x - top);
                l = fmaf(ml.y, keep, l);
                x = fmaf(ws_o[i * D + ch], keep, x);
            }
        s_x[part][ch] = x;
        if (ch == 0) s_l[part] = l;
        __syncthreads();
        x = l = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            x += s_x[i][ch];
            l += s_l[i];
        }
        y = x / l;
        lse = top * kLn2 + logf(l);
    }
    if (part != 0) return;
    if (a.out_bf16)
        store_one(static_cast<__nv_bfloat16*>(a.out) + r * D + ch, y);
    else
        store_one(static_cast<float*>(a.out) + r * D + ch, y);
    if (ch == 0 && a.lse != nullptr) a.lse[r] = lse;
}

// Query heads per warp: the smallest of 1, 2, 4, 8 that covers the group, or 8
// with several chunks of warps.
int chunk_heads(int G) { return G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : 8; }

DecodeShape simple_shape(const DecodeArgs& a, int* chunks)
{
    const int G = a.Hq / a.Hk, gt = chunk_heads(G);
    int c = 1;
    while (c * gt < G && c < NW) c *= 2;
    *chunks = c;
    DecodeShape s;
    s.heads = c * gt;
    s.units = a.Hk * ((G + s.heads - 1) / s.heads);
    s.ctas = sm_count() * 2;
    s.tile_shift = kTileShift;
    return s;
}

template <int D>
cudaError_t launch_simple(const DecodeArgs& a, const DecodeShape& s, int chunks, cudaStream_t st)
{
    switch (chunk_heads(a.Hq / a.Hk)) {
        case 1: paged_decode_kernel<D, 1><<<s.ctas, NT, 0, st>>>(a, s, chunks); break;
        case 2: paged_decode_kernel<D, 2><<<s.ctas, NT, 0, st>>>(a, s, chunks); break;
        case 4: paged_decode_kernel<D, 4><<<s.ctas, NT, 0, st>>>(a, s, chunks); break;
        default: paged_decode_kernel<D, 8><<<s.ctas, NT, 0, st>>>(a, s, chunks);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_join(const DecodeArgs& a, const DecodeShape& s, cudaStream_t stream)
{
    const int64_t rows = (int64_t)a.N * a.Hq;
    return launch_after(a.D == 64 ? decode_join_kernel<64> : decode_join_kernel<128>,
                        (unsigned)rows, NT, stream, a, s);
}

int64_t paged_decode_workspace_bytes(int32_t N, int32_t Hq, int32_t Hk, int32_t D)
{
    DecodeArgs a = {};
    a.N = N; a.Hq = Hq; a.Hk = Hk; a.D = D;
    int chunks;
    int64_t most = 0;
    for (const DecodeShape& s : {simple_shape(a, &chunks), decode_tc_shape(a)}) {
        const int64_t b = decode_o_offset(N, s) + (int64_t)2 * s.ctas * s.heads * D * 4;
        if (b > most) most = b;
    }
    return most;
}

cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t stream)
{
    cudaError_t e;
    DecodeShape s;
    if (a.bf16) {
        s = decode_tc_shape(a);
        e = launch_paged_decode_tc(a, s, stream);
    } else {
        int chunks;
        s = simple_shape(a, &chunks);
        e = a.D == 64 ? launch_simple<64>(a, s, chunks, stream)
                      : launch_simple<128>(a, s, chunks, stream);
    }
    return e == cudaSuccess ? launch_decode_join(a, s, stream) : e;
}

}  // namespace kda
