// kda_paged_decode for FP32 caches, on CUDA cores (IEEE FP32 products), and the join
// of split rows for either type.
//
//     s_t = scale q . k_t,   out = sum e^(s_t) v_t / sum e^(s_t)
//
// HBM-bound: every k and v is read once, 2 D values a token and key-value head.
// One CTA per SM; two producer warps (keys, values) fill slots of 32 tokens (64 of 64
// channels) by TMA, one box per page (the keys in 128-byte columns, swizzled, so that
// 32 lanes can read 32 rows without bank conflicts).  Six slots of 32 KB (five with units of
// 16 heads of 64 channels) have a warp each, or two that share the heads, which takes its tile
// on its own:
//   scores   a lane has 1 to 8 tokens and the unit's heads or a quarter of them (so that a
//            value read from shared memory is used four times and more), queries scaled
//            by scale * log2 e beforehand, products in pairs (f32x2);
//   softmax  a reduction over the lanes per head; the reference maximum moves only when it
//            would grow by more than 2^8, which is exact and rarely rescales;
//   values   four channels a lane, the weights back from shared memory four tokens
//            at a time.  Rows past the end are not read.
// No lane reduces anything else across the warp.  At the end of a
// row the warps merge (m, l, o) through shared memory, four heads at a time.
//
// Measured: 16 requests of 1 to 4096 tokens, 16 heads of 64 channels with their own keys,
// 50 us, 84% of the rate of a plain copy (start, row ends and join are the rest).  Groups
// of 8 heads reach 79 to 82%, of 16 heads 51%, of 32 heads (two units that each read the
// cache) 28%: there the reads of shared memory bound the kernel (32 requests of 4096 tokens: 76
// to 81% of its wavefronts, the FMA pipe 23%, the issue slots 39%).
#include <cuda_runtime.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "kda_paged_sched.cuh"
#include "kda_paged_tma.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kJoin = 256;             // threads of the join
constexpr float kGrowth = 8.f;         // log2 of the growth that moves the reference maximum
constexpr int kMerge = 4;              // heads merged at a time

template <int D, int GT> struct Cfg {
    static constexpr int W = D == 64 && GT == 16 ? 5 : 6;     // slots
    static constexpr int PARTS = GT >= 8 ? 2 : 1, GH = GT / PARTS;   // warps per slot, heads of each
    static constexpr int CW = W * PARTS;                       // warps that compute
    static constexpr int NT = 32 * (CW + 2);
    static constexpr int kTile = 4096 / D;                     // tokens per tile
    // a warp's lanes for the scores: HS groups, each for HG heads, TT tokens a lane
    static constexpr int HS = GH >= 8 ? 4 : GH == 4 ? 2 : 1, HG = GH / HS, TL = 32 / HS, TT = kTile / TL;
    static constexpr int kTileShift = D == 128 ? 5 : 6;
    static constexpr uint32_t TILE = kTile * D * 4;            // keys or values of a slot
    static constexpr uint32_t SLOT = 2 * TILE;
    static constexpr uint32_t OFF_Q = W * SLOT, OFF_P = OFF_Q + GT * D * 4,
                              OFF_O = OFF_P + W * GT * kTile * 4,
                              OFF_ML = OFF_O + W * kMerge * D * 4, OFF_BAR = OFF_ML + W * GT * 8,
                              SMEM = OFF_BAR + 512 + 1024;
    static_assert(SMEM + 256 <= 227 * 1024 && 2 * W * 8 + 4 <= 512, "shared memory of a CTA");
};

struct Maps {
    CUtensorMap k, v;
};

struct Bars {
    uint64_t full[6], empty[6];        // slots
    int32_t abort;
};

template <int D, int GT>
__global__ void __launch_bounds__(Cfg<D, GT>::NT, 1)
paged_decode_kernel(DecodeArgs a, DecodeShape sh, const __grid_constant__ Maps maps)
{
    using C = Cfg<D, GT>;
    constexpr int W = C::W, kTile = C::kTile, kTileShift = C::kTileShift;
    constexpr int PARTS = C::PARTS, GH = C::GH, CW = C::CW, HG = C::HG, TL = C::TL, TT = C::TT;
    constexpr int BLOCKS = D / 32;                 // 128-byte columns of a key row
    constexpr int LPR = D / 4, RPW = 32 / LPR;     // lanes per value row, rows at a time
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    Bars& bar = *reinterpret_cast<Bars*>(sm + C::OFF_BAR);
    float* s_q = reinterpret_cast<float*>(sm + C::OFF_Q);          // [GT][D]
    float* s_p = reinterpret_cast<float*>(sm + C::OFF_P);          // [CW][GH][kTile]
    float* s_o = reinterpret_cast<float*>(sm + C::OFF_O);          // [W][kMerge][D]
    float2* s_ml = reinterpret_cast<float2*>(sm + C::OFF_ML);      // [W][GT]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.Hq / a.Hk, groups = sh.units / a.Hk;

    if (tid == 0) {
        for (int i = 0; i < W; ++i) {
            mbar_init(&bar.full[i], 2);
            mbar_init(&bar.empty[i], PARTS);
        }
        bar.abort = 0;
        fence_mbar_init();
    }
    wait_for_previous();
    DecodeLens lens;
    lens.load(a);
    __syncthreads();                               // the barriers
    char* ws = static_cast<char*>(a.workspace);
    const DecodeRange rg = decode_range<C::NT>(a, sh, lens, ws);

    BoundedWait wait(&bar.abort, a.status);
    DecodeWalk w(rg, a, sh, groups);
    if (warp >= CW) {
        // ------------------------------------------------------------ producers
        const bool keys = warp == CW;
        const void* map = keys ? &maps.k : &maps.v;
        const int shift = a.page_shift < kTileShift ? a.page_shift : kTileShift;
        const int rows = 1 << shift;                               // tokens per box
        const int token = (keys ? lane / BLOCKS : lane) << shift, col = keys ? lane % BLOCKS : 0;
        const uint32_t box = keys ? col * (kTile * 128) + token * 128 : C::TILE + token * (D * 4);
        uint32_t c = 0;
        int t = 0;
        DecodeTile tile;
        bool more = tile.next(w, t, a, sh, kTile, shift, token);
        for (; more; ++c, more = tile.next(w, t, a, sh, kTile, shift, token)) {
            const uint32_t slot = c % W;
            wait(&bar.empty[slot], ((c / W) & 1) ^ 1);
            wait.dead = __any_sync(0xffffffffu, wait.dead);
            if (wait.dead) break;
            if (lane == 0) mbar_arrive_expect_tx(&bar.full[slot], tile.boxes * rows * D * 4);
            __syncwarp();
            if (token < tile.boxes << shift)
                tma_load_2d(smem_u32(sm + slot * C::SLOT) + box, map, 32 * col,
                            page_row(a, tile.entry, tile.hk, tile.at), &bar.full[slot]);
        }
        // every copy has landed before the CTA ends
        if (lane == 0)
            for (uint32_t i = c > (uint32_t)W ? c - W : 0; i < c; ++i)
                mbar_wait(&bar.full[i % W], (i / W) & 1);
        return;
    }
    // ---------------------------------------------------------------- compute
    const float qscale = a.scale * kLog2e;
    float2* ws_ml = reinterpret_cast<float2*>(ws + decode_ml_offset(sh));
    float* ws_o = reinterpret_cast<float*>(ws + decode_o_offset(sh));
    float* my_p = s_p + warp * GH * kTile;
    const int mine = warp % W, first = warp / W * GH;              // the warp's slot and heads
    const int sub = lane / LPR, chan = (lane % LPR) * 4;           // for the values
    const int head = lane / TL * HG, tl = lane % TL;               // for the scores
    uint32_t c0 = 0;                               // the CTA's tiles before this row
    while (w.next(a, sh)) {
        const int hk = w.hk, g0 = w.part * GT;                         // in the group of G
        for (int i = tid; i < GT * D; i += 32 * CW) {
            const int g = i / D;
            s_q[i] = g0 + g < G ? static_cast<const float*>(a.q)[((int64_t)w.n * a.Hq + hk * G + g0) *
                                                                     D + i] * qscale
                                : 0.f;
        }
        float m[HG], l[HG], o[GH][4];
#pragma unroll
        for (int g = 0; g < HG; ++g) {
            m[g] = -CUDART_INF_F;
            l[g] = 0.f;
        }
#pragma unroll
        for (int g = 0; g < GH; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[g][i] = 0.f;
        named_sync(1, 32 * CW);
        // tile c of the CTA is in slot c % W, which is the warp's own: a warp that shared
        // slots could mistake an earlier filling's phase for its own
        for (int t = w.tile0 + (int)((mine + W - c0 % W) % W); t < w.tile1; t += W) {
            const uint32_t c = c0 + (t - w.tile0);
            const int valid = min(kTile, w.L - (t << kTileShift));
            wait(&bar.full[mine], (c / W) & 1);
            // tokens tl, tl + TL, ...: their rows have the same place in the swizzle
            const unsigned char* kt = sm + mine * C::SLOT + tl * 128;
            const float* vt = reinterpret_cast<const float*>(sm + mine * C::SLOT + C::TILE);
            float2 s[TT][HG];
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int g = 0; g < HG; ++g) s[i][g] = make_float2(0.f, 0.f);
#pragma unroll(TT * HG > 16 ? 2 : 4)
            for (int j = 0; j < D / 4; ++j) {
                float4 k[TT];
#pragma unroll
                for (int i = 0; i < TT; ++i)
                    k[i] = *reinterpret_cast<const float4*>(kt + (j >> 3) * (kTile * 128) + i * TL * 128 +
                                                            (((j & 7) ^ (tl & 7)) << 4));
#pragma unroll
                for (int g = 0; g < HG; ++g) {
                    const float4 q = *reinterpret_cast<const float4*>(s_q + (first + head + g) * D + 4 * j);
#pragma unroll
                    for (int i = 0; i < TT; ++i) {
                        s[i][g] = fma2(make_float2(q.x, q.y), make_float2(k[i].x, k[i].y), s[i][g]);
                        s[i][g] = fma2(make_float2(q.z, q.w), make_float2(k[i].z, k[i].w), s[i][g]);
                    }
                }
            }
            __syncwarp();                          // the last tile's weights are read
            float x[TT][HG], top[HG];
            bool grown = false;
#pragma unroll
            for (int g = 0; g < HG; ++g) {
                top[g] = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    x[i][g] = tl + TL * i < valid ? s[i][g].x + s[i][g].y : -CUDART_INF_F;
                    top[g] = fmaxf(top[g], x[i][g]);
                }
                if constexpr (TL == 32) {
                    top[g] = warp_max(top[g]);
                } else {
#pragma unroll
                    for (int k = TL / 2; k > 0; k >>= 1)
                        top[g] = fmaxf(top[g], __shfl_xor_sync(0xffffffffu, top[g], k));
                }
                grown |= top[g] > m[g] + kGrowth;
            }
            if (__any_sync(0xffffffffu, grown)) {
                float keep[HG];
#pragma unroll
                for (int g = 0; g < HG; ++g) {
                    keep[g] = 1.f;
                    if (top[g] > m[g] + kGrowth) {
                        keep[g] = exp2f(m[g] - top[g]);
                        m[g] = top[g];
                    }
                    l[g] *= keep[g];
                }
#pragma unroll
                for (int g = 0; g < GH; ++g) {
                    const float k = __shfl_sync(0xffffffffu, keep[g % HG], g / HG * TL);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[g][i] *= k;
                }
            }
#pragma unroll
            for (int g = 0; g < HG; ++g) {
                // all scores so far -infinity: nothing to subtract
                const float ref = m[g] == -CUDART_INF_F ? 0.f : m[g];
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    const float e = exp2f(x[i][g] - ref);
                    l[g] += e;
                    my_p[(head + g) * kTile + tl + TL * i] = e;
                }
            }
            __syncwarp();
#pragma unroll
            for (int r = 0; r < kTile; r += 4 * RPW) {
                if (r >= valid) break;             // uniform
                float4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = r + 4 * sub + i;
                    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);    // 0 * NaN is not 0
                    if (row < valid) v[i] = *reinterpret_cast<const float4*>(vt + row * D + chan);
                }
#pragma unroll
                for (int g = 0; g < GH; ++g) {
                    const float4 p = *reinterpret_cast<const float4*>(my_p + g * kTile + r + 4 * sub);
                    const float pi[4] = {p.x, p.y, p.z, p.w};
                    float2 lo = make_float2(o[g][0], o[g][1]), hi = make_float2(o[g][2], o[g][3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        lo = fma2(both(pi[i]), make_float2(v[i].x, v[i].y), lo);
                        hi = fma2(both(pi[i]), make_float2(v[i].z, v[i].w), hi);
                    }
                    o[g][0] = lo.x;
                    o[g][1] = lo.y;
                    o[g][2] = hi.x;
                    o[g][3] = hi.y;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.empty[mine]);
        }
        // merge: the row's maximum of each head over the warps, then outputs to it; in the
        // order of the row's tiles, whatever the CTA did before
        const int turn = c0 % W;                       // the warp of the row's first tile
        c0 += w.tile1 - w.tile0;
#pragma unroll
        for (int g = 0; g < HG; ++g) {
#pragma unroll
            for (int k = TL / 2; k > 0; k >>= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], k);
            if (tl == 0) s_ml[mine * GT + first + head + g] = make_float2(m[g], l[g]);
        }
        named_sync(1, 32 * CW);
        const bool whole = w.tile0 == 0 && w.tile1 == w.tiles;
        const int64_t r0 = whole ? (int64_t)w.n * a.Hq + hk * G + g0
                                 : (2 * (int64_t)blockIdx.x + (w.tile0 == 0)) * GT;
#pragma unroll
        for (int gb = 0; gb < GT; gb += kMerge) {
            // the warps that have these heads
            if (first == gb / GH * GH) {
#pragma unroll
                for (int g = gb; g < gb + kMerge && g < GT; ++g) {
                    float top = -CUDART_INF_F;
#pragma unroll
                    for (int k = 0; k < W; ++k) top = fmaxf(top, s_ml[k * GT + g].x);
                    const float keep = top == -CUDART_INF_F ? 0.f : exp2f(s_ml[mine * GT + g].x - top);
                    float (&x)[4] = o[g % GH];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] *= keep;
#pragma unroll
                        for (int k = LPR; k < 32; k <<= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], k);
                    }
                    if (sub == 0)
                        *reinterpret_cast<float4*>(s_o + (mine * kMerge + g - gb) * D + chan) =
                            make_float4(x[0], x[1], x[2], x[3]);
                }
            }
            named_sync(1, 32 * CW);
            for (int i = tid; i < kMerge * D; i += 32 * CW) {
                const int g = gb + i / D, ch = i % D;
                if (g >= GT || g0 + g >= G) continue;
                float top = -CUDART_INF_F, sum = 0.f, x = 0.f;
#pragma unroll
                for (int k = 0; k < W; ++k) top = fmaxf(top, s_ml[k * GT + g].x);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int k = turn + j < W ? turn + j : turn + j - W;
                    const float2 ml = s_ml[k * GT + g];
                    // without a maximum the sums are zero, or NaN where scores are
                    sum += top == -CUDART_INF_F ? ml.y : ml.y * exp2f(ml.x - top);
                    x += s_o[(k * kMerge + g - gb) * D + ch];
                }
                const int64_t r = r0 + g;
                if (whole) {
                    const float y = x / sum;
                    if (a.out_bf16)
                        store_one(static_cast<__nv_bfloat16*>(a.out) + r * D + ch, y);
                    else
                        store_one(static_cast<float*>(a.out) + r * D + ch, y);
                    if (ch == 0 && a.lse != nullptr) a.lse[r] = top * kLn2 + logf(sum);
                } else {
                    ws_o[r * D + ch] = x;
                    if (ch == 0) ws_ml[r] = make_float2(top, sum);
                }
            }
            named_sync(1, 32 * CW);
        }
    }
}

// Joins the split rows.  Block (b, y) joins the row whose first split is where CTA b's
// tiles begin, every gridDim.y-th head from y; most blocks find nothing to do.  Four
// channels a lane; the block's groups of D / 4 lanes take a head each, or, where the
// row has many pieces, share the pieces of one head, four at a time each.  The order of
// the sums is set by the number of pieces alone.  Empty requests' rows are dealt to all
// blocks.
template <int D>
__global__ void __launch_bounds__(kJoin) decode_join_kernel(DecodeArgs a, DecodeShape sh)
{
    constexpr int LANES = D / 4, P = kJoin / LANES;        // lanes of a group, groups
    constexpr int kMany = 4;       // pieces requested together, and from which groups share a head
    __shared__ float4 s_x[P][LANES];
    __shared__ float2 s_ml[P];
    const int ch = (threadIdx.x % LANES) * 4, part = threadIdx.x / LANES;
    auto store = [&](int64_t r, float4 y) {
        if (a.out_bf16)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + r * D + ch) =
                make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + r * D + ch) = y;
    };
    wait_for_previous();
    for (int64_t n = blockIdx.x + (int64_t)gridDim.x * blockIdx.y; n < a.N;
         n += (int64_t)gridDim.x * gridDim.y) {
        if (decode_len(a, n) != 0) continue;
        for (int h = part; h < a.Hq; h += P) {
            store(n * a.Hq + h, make_float4(0.f, 0.f, 0.f, 0.f));
            if (ch == 0 && a.lse != nullptr) a.lse[n * a.Hq + h] = -CUDART_INF_F;
        }
    }
    const char* ws = static_cast<const char*>(a.workspace);
    const DecodeSplit st = reinterpret_cast<const DecodeSplit*>(ws)[blockIdx.x];
    const int pieces = st.last - st.first + 1;
    if (pieces <= 0) return;
    const float2* ws_ml = reinterpret_cast<const float2*>(ws + decode_ml_offset(sh));
    const float* ws_o = reinterpret_cast<const float*>(ws + decode_o_offset(sh));
    const int G = a.Hq / a.Hk, groups = sh.units / a.Hk;
    const int hk = st.u / groups, g0 = (st.u - hk * groups) * sh.heads;
    const int heads = min(sh.heads, G - g0);
    const bool share = pieces >= kMany;
    const int stride = share ? P : 1, first = share ? part : 0;
    for (int gb = share ? blockIdx.y : blockIdx.y * P; gb < heads;
         gb += share ? gridDim.y : gridDim.y * P) {
        const int g = share ? gb : gb + part;
        // piece i: the row begins in the first CTA's tiles
        auto piece = [&](int i) { return (2 * (int64_t)(st.first + i) + (i == 0)) * sh.heads + g; };
        // the maxima, sums and outputs of up to kMany pieces are requested together
        float top = -CUDART_INF_F, l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float2 (&ml)[kMany], const float4 (&o)[kMany]) {
            float m = top;
#pragma unroll
            for (int j = 0; j < kMany; ++j) m = fmaxf(m, ml[j].x);
            if (m == -CUDART_INF_F) {
                // no score but -infinity and NaN so far: sums of zero, or NaN
#pragma unroll
                for (int j = 0; j < kMany; ++j) l += ml[j].y;
                return;
            }
            const float old = exp2f(top - m);
            top = m;
            l *= old;
            x = make_float4(x.x * old, x.y * old, x.z * old, x.w * old);
#pragma unroll
            for (int j = 0; j < kMany; ++j) {
                const float keep = exp2f(ml[j].x - m);
                l = fmaf(ml[j].y, keep, l);
                x.x = fmaf(o[j].x, keep, x.x);
                x.y = fmaf(o[j].y, keep, x.y);
                x.z = fmaf(o[j].z, keep, x.z);
                x.w = fmaf(o[j].w, keep, x.w);
            }
        };
        for (int i0 = first; i0 < pieces && g < heads; i0 += kMany * stride) {
            float2 ml[kMany];
            float4 o[kMany];
#pragma unroll
            for (int j = 0; j < kMany; ++j) {
                const int i = i0 + j * stride;
                ml[j] = make_float2(-CUDART_INF_F, 0.f);
                o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < pieces) {
                    ml[j] = ws_ml[piece(i)];
                    o[j] = *reinterpret_cast<const float4*>(ws_o + piece(i) * D + ch);
                }
            }
            add(ml, o);
        }
        if (share) {
            __syncthreads();                               // the last head's sums are read
            s_x[part][ch / 4] = x;
            if (ch == 0) s_ml[part] = make_float2(top, l);
            __syncthreads();
            if (part != 0) continue;
            for (int i0 = 1; i0 < P; i0 += kMany) {
                float2 ml[kMany];
                float4 o[kMany];
#pragma unroll
                for (int j = 0; j < kMany; ++j) {
                    const bool any = i0 + j < P;
                    ml[j] = any ? s_ml[i0 + j] : make_float2(-CUDART_INF_F, 0.f);
                    o[j] = any ? s_x[i0 + j][ch / 4] : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                add(ml, o);
            }
        }
        if (g >= heads) continue;
        const float inv = 1.f / l;
        const int64_t r = (int64_t)st.n * a.Hq + hk * G + g0 + g;
        store(r, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
        if (ch == 0 && a.lse != nullptr) a.lse[r] = top * kLn2 + logf(l);
    }
}

// Query heads per unit: the smallest of 1, 2, 4, 8, 16 that covers the group (more
// heads than that read the cache once per 16).
int unit_heads(int G) { return G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : G <= 8 ? 8 : 16; }

DecodeShape fp32_shape(const DecodeArgs& a)
{
    const int G = a.Hq / a.Hk;
    DecodeShape s;
    s.heads = unit_heads(G);
    s.units = a.Hk * ((G + s.heads - 1) / s.heads);
    s.ctas = sm_count();
    s.tile_shift = a.D == 128 ? 5 : 6;
    // A row's end (the warps' partly filled rounds, the merge) costs as much as 192 tokens,
    // with several heads to merge 256: heads of 128 channels and 96 / 192 / 256 / 320 tokens,
    // 103 requests of 1 to 863 with 8 heads a group 119, 94.5, 93.0, 93.1 us, 32 of 1 to 2000
    // with 4 heads 67, 55.5, 52.6, 52.7, 64 of 1 to 256 with one head 22.3, 21.6, 22.5, 22.3.
    s.start = (s.heads >= 4 ? 256 : 192) >> s.tile_shift;
    return s;
}

template <int D, int GT>
cudaError_t launch_typed(const DecodeArgs& a, const DecodeShape& s, cudaStream_t stream)
{
    using C = Cfg<D, GT>;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    const int page = 1 << a.page_shift, box = page < C::kTile ? page : C::kTile;
    const int64_t rows = (int64_t)a.num_pages * a.Hk * page, qrows = (int64_t)a.N * a.Hq;
    // an empty cache has no page to read: the maps only have to be valid
    cudaError_t e = encode_rows(&maps.k, rows ? a.k : a.q, false, rows ? rows : qrows, D, 32, box, true);
    if (e == cudaSuccess)
        e = encode_rows(&maps.v, rows ? a.v : a.q, false, rows ? rows : qrows, D, D, box, false);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> set{0};
    e = allow_smem(paged_decode_kernel<D, GT>, C::SMEM, &set);
    if (e != cudaSuccess) return e;
    return launch_after(paged_decode_kernel<D, GT>, launch_config(s.ctas, C::NT, C::SMEM), stream, a, s,
                        maps);
}

template <int D>
cudaError_t launch_fp32(const DecodeArgs& a, const DecodeShape& s, cudaStream_t st)
{
    switch (s.heads) {
        case 1: return launch_typed<D, 1>(a, s, st);
        case 2: return launch_typed<D, 2>(a, s, st);
        case 4: return launch_typed<D, 4>(a, s, st);
        case 8: return launch_typed<D, 8>(a, s, st);
        default: return launch_typed<D, 16>(a, s, st);
    }
}

}  // namespace

cudaError_t launch_decode_join(const DecodeArgs& a, const DecodeShape& s, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = launch_config(s.ctas, kJoin);
    // many blocks for a head's pieces each only where rows are few and the pieces many
    const int64_t rows = (int64_t)a.N * s.units;
    const int heads = s.heads < 8 ? s.heads : 8;
    cfg.gridDim = dim3((unsigned)s.ctas, (unsigned)(rows * 2 < s.ctas ? heads : heads < 2 ? 1 : 2));
    return launch_after(a.D == 64 ? decode_join_kernel<64> : decode_join_kernel<128>, cfg, stream, a,
                        s);
}

int64_t paged_decode_workspace_bytes(int32_t N, int32_t Hq, int32_t Hk, int32_t D)
{
    DecodeArgs a = {};
    a.N = N; a.Hq = Hq; a.Hk = Hk; a.D = D;
    int64_t most = 0;
    for (const DecodeShape& s : {fp32_shape(a), decode_tc_shape(a)}) {
        const int64_t b = decode_workspace(s, D);
        if (b > most) most = b;
    }
    return most;
}

cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t stream)
{
    const DecodeShape s = a.bf16 ? decode_tc_shape(a) : fp32_shape(a);
    const cudaError_t e = a.bf16 ? launch_paged_decode_tc(a, s, stream)
                          : a.D == 64 ? launch_fp32<64>(a, s, stream)
                                      : launch_fp32<128>(a, s, stream);
    return e == cudaSuccess ? launch_decode_join(a, s, stream) : e;
}

}  // namespace kda
