// Backward of attention for several tokens, BF16 on the tensor cores (tcgen05), in two
// kernels that each form the scores again:
//
//   keys     a CTA has 128 keys of a sequence and one key-value head, and walks over the rows
//            (tokens times the group's heads) that see them, 128 at a time:
//                S^T = K Q^T, dP^T = V dO^T          both operands in shared memory
//                dV += P^T dO, dK += dS^T Q          P^T and dS^T in tensor memory
//   queries  a CTA has 128 rows and walks over the key tiles they see:
//                S = Q K^T, dP = dO V^T, dQ += dS K
//
// so that every gradient adds up in one CTA's tensor memory, over all heads of the group, in
// an order that the sizes set: no atomics, the same bits every time.  The price is seven
// products a tile of scores instead of five.  Transposing the scores in the first kernel lets
// P and dS stay in tensor memory as operands; the other operand of every product is read from
// shared memory as TMA left it, as rows or as columns.
//
// Eight warps form P and dS, a thread half a row of a tile: P while the tensor core works on
// the products with the tile before, dS = P (dP - delta) while it forms P^T dO and the next
// scores.  P and dS are rounded to BF16 (2^-8) as operands.  Rows with few keys
// have the largest dS and lose most to the rounding of `out` in delta: in a tile of rows that
// sees one tile of keys (up to 128 for its last row) delta is the sum of P dP in FP32, which the
// second kernel forms (it runs first) and leaves to the other, and both take dS as two BF16
// parts, the second in columns of dP that the first leaves free
// (sequences of 1 to 700 tokens: dq and dk 2.5e-3 off without both; of 2 to 4 tokens 3.1e-3 off with
// the rounded out; the rounding of the result is 1.7e-3).
// A warp reads the rows' lse and delta.
//
// Bound by the tensor pipe in long sequences: one of 8192 tokens, 64 / 8 heads of 128 channels,
// takes 1.28 ms for dk and dv and 0.91 for dq (1720 and 1820 TFLOP/s of the 1898 that a library
// product reaches, counting the products made), delta 0.04.  Short ones are bound by a tile's start
// and end: 8 sequences of 1 to 2048 tokens 257, 222 and 36 us.  What lies between the
// products on the issuing warp counts: the same loops with conditions between them took 1.32 and
// 1.05 ms, dq with one buffer of dP and a CTA a tile 1.25.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "kda_attn_tc.cuh"

namespace kda {
namespace {

using namespace tc;

template <int D> struct Cfg {
    static constexpr int HALVES = D / 64;
    static constexpr uint32_t TILE = 128 * D * 2;              // 128 rows of keys, values, queries or dO
    static constexpr uint32_t OFF_RING = 2 * TILE;             // two stages of two tiles
    static constexpr uint32_t OFF_STAT = OFF_RING + 4 * TILE, OFF_BAR = OFF_STAT + 2 * 1024,
                              SMEM = OFF_BAR + 512 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
    static constexpr int NT = 352, WARP_LOAD = 8, WARP_MMA = 9, WARP_STAT = 10;
};

struct KvMaps {
    CUtensorMap q, dout, k, v;
};
struct QMaps {
    CUtensorMap q, dout, k, v, dq;
};

struct Bars {
    uint64_t afull[2];                 // the CTA's own two tiles
    uint64_t full[2][2], empty[2][2];  // the walked tiles: [first or second][stage]
    uint64_t sfull, pfull;             // S, P in its place
    uint64_t dpfull, dsfull;           // dP, dS in its place
    uint64_t statfull[2], statempty[2];
    uint64_t done;
    uint32_t tmem;
    int32_t abort;
    int32_t found;
    AttnTile tile;
};

__device__ __forceinline__ void start(Bars& bar, const AttnArgs& a, int32_t item, int32_t tokens)
{
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.afull[i], 1);
            for (int x = 0; x < 2; ++x) {
                mbar_init(&bar.full[x][i], 1);
                mbar_init(&bar.empty[x][i], 1);
            }
            mbar_init(&bar.statfull[i], 1);
            mbar_init(&bar.statempty[i], 8);
        }
        mbar_init(&bar.sfull, 1);
        mbar_init(&bar.pfull, 8);
        mbar_init(&bar.dpfull, 1);
        mbar_init(&bar.dsfull, 8);
        mbar_init(&bar.done, 1);
        bar.abort = 0;
        fence_mbar_init();
    }
    wait_for_previous();
    const bool bad = a.N > kAttnOrdered && attn_bad(a);
    if (warp == 0) {
        AttnTile t;
        const bool found = attn_find(a, bad, item, tokens, kTcKeyShift, t);
        if (tid == 0) {
            bar.tile = t;
            bar.found = found;
        }
    } else if (warp == 9) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
}

// Zeroes rows first .. last - 1 of a tile, by `threads` threads, for the products' reads.
template <int D>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int first, int last, int thread, int threads)
{
    constexpr int HALVES = D / 64;
    for (int e = thread; e < (last - first) * 8 * HALVES; e += threads)
        *reinterpret_cast<uint4*>(tile + (e >> 3) % HALVES * (128 * 128) + (first + (e >> 3) / HALVES) * 128 +
                                  (e & 7) * 16) = make_uint4(0, 0, 0, 0);
}

// 64 values of a thread's lane, from column `t` on, as BF16 pairs in 32 columns there.
__device__ __forceinline__ void store_pairs(uint32_t t, const float (&x)[64])
{
    uint32_t u[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    tmem_st32(t, u);
    tmem_st_wait();
}

// What the BF16 pairs of store_pairs leave of the values, as BF16 pairs in the 32 columns
// behind theirs.
__device__ __forceinline__ void store_rests(uint32_t t, const float (&x)[64])
{
    uint32_t u[32];
    auto rest = [](float v, uint32_t bits) {
        return fabsf(v) < CUDART_INF_F ? v - __uint_as_float(bits) : 0.f;
    };
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint32_t p = pack_bf16(x[2 * i], x[2 * i + 1]);
        u[i] = pack_bf16(rest(x[2 * i], p << 16), rest(x[2 * i + 1], p & 0xffff0000u));
    }
    tmem_st32(t + 32, u);
}

// A lane's D values, scaled, to a row of the output.
template <int D> __device__ __forceinline__ void store_row(uint32_t t, float scale, bool live, __nv_bfloat16* y)
{
#pragma unroll
    for (int c = 0; c < D; c += 32) {
        float x[32];
        __syncwarp();
        tmem_ld32(t + c, x);
        if (live) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
                *reinterpret_cast<uint4*>(y + c + i) = make_uint4(
                    pack_bf16(x[i] * scale, x[i + 1] * scale), pack_bf16(x[i + 2] * scale, x[i + 3] * scale),
                    pack_bf16(x[i + 4] * scale, x[i + 5] * scale), pack_bf16(x[i + 6] * scale, x[i + 7] * scale));
        }
    }
}

// ---------------------------------------------------------------- dk, dv
template <int D>
__global__ void __launch_bounds__(Cfg<D>::NT, 1)
attn_bwd_kv_tc_kernel(AttnArgs a, AttnShape sh, const __grid_constant__ KvMaps maps)
{
    using C = Cfg<D>;
    constexpr int HALVES = C::HALVES;
    constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 256 + D;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    Bars& bar = *reinterpret_cast<Bars*>(sm + C::OFF_BAR);
    static_assert(sizeof(Bars) <= 512, "barriers");
    float* stats = reinterpret_cast<float*>(sm + C::OFF_STAT);     // [stage][-lse log2 e, -delta][128]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t hk = blockIdx.x % a.Hk, item = blockIdx.x / a.Hk, rows = sh.tokens * sh.heads;
    // Rows of a tile that no copy fills are zeros for good.
    if (rows < 128) {
        for (int x = 0; x < 4; ++x) zero_rows<D>(sm + C::OFF_RING + x * C::TILE, rows, 128, tid, C::NT);
        fence_async_smem();
    }
    start(bar, a, item, kTcKeys);
    const uint32_t tmem = uniform(bar.tmem);
    BoundedWait wait(&bar.abort, a.status);
    if (uniform(bar.found)) {
        const AttnTile t = bar.tile;
        // the tile found has t.index tiles of queries before it; the one with as many behind it
        const int32_t nt = (t.seq_tokens + kTcKeys - 1) >> kTcKeyShift, key0 = (nt - 1 - t.index) << kTcKeyShift;
        const int32_t left = uniform(t.seq_tokens - key0);         // tokens from the first key on
        const int32_t per = uniform((left + sh.tokens - 1) / sh.tokens), n = per * sh.parts;
        const int32_t last = left - (per - 1) * sh.tokens;         // tokens of a part's last tile
        auto ring = [&](int x, int32_t i) { return sm + C::OFF_RING + ((i & 1) * 2 + x) * C::TILE; };
        // whether tile `at` of a part takes dS in two parts: where the other kernel's tile has one
        // tile of keys
        auto in_two = [&](int32_t at) { return key0 == 0 && min((at + 1) * sh.tokens, left) <= kTcKeys; };

        if (warp == C::WARP_LOAD) {
            // -------------------------------------------------------- producer
            if (lane == 0) {
                for (int x = 0; x < 2; ++x) {
                    mbar_arrive_expect_tx(&bar.afull[x], C::TILE);
                    for (int h = 0; h < HALVES; ++h)
                        tma_load_3d(sm + x * C::TILE + h * (128 * 128), x ? &maps.v : &maps.k, 64 * h, hk,
                                    t.seq0 + key0, &bar.afull[x]);
                }
                int32_t part = 0, at = 0, loads[2] = {0, 0};       // copies of each ring
                for (int32_t i = 0; i < n; ++i) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        wait(&bar.empty[x][i & 1], ((i >> 1) & 1) ^ 1);
                        if (wait.dead) break;
                        ++loads[x];
                        mbar_arrive_expect_tx(&bar.full[x][i & 1], (uint32_t)rows * 128 * HALVES);
                        for (int h = 0; h < HALVES; ++h)
                            tma_load_3d(ring(x, i) + h * (128 * 128), x ? &maps.dout : &maps.q, 64 * h,
                                        (hk * sh.parts + part) * sh.heads, t.seq0 + key0 + at * sh.tokens,
                                        &bar.full[x][i & 1]);
                    }
                    if (wait.dead) break;
                    if (++at == per) {
                        at = 0;
                        ++part;
                    }
                }
                // every copy has landed before the CTA ends
                mbar_wait(&bar.afull[0], 0);
                mbar_wait(&bar.afull[1], 0);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    for (int32_t k = max(0, loads[x] - 2); k < loads[x]; ++k)
                        mbar_wait(&bar.full[x][k & 1], (k >> 1) & 1);
            }
        } else if (warp == C::WARP_MMA) {
            // -------------------------------------------------------- MMA
            {
                const uint32_t lead = elect_one();
                const bool withhold = a.fault == KDA_TEST_FAULT_ATTENTION_BWD_KV && blockIdx.x == 0;
                WarpWait wait(&bar.abort, a.status);
                constexpr uint32_t id_s = idesc(kFmtBF16, 128, 128), id_d = idesc(kFmtBF16, 128, D, false, true);
                const uint32_t base = smem_u32(sm);
                const uint64_t dA = desc_kmajor(base, 128, 0), dB = desc_kmajor(base + C::OFF_RING, 128, 0);
                const uint64_t dN = D == 128 ? desc_mnmajor128(base + C::OFF_RING, 128 * 128, 0)
                                             : desc_mnmajor64(base + C::OFF_RING, 0);
                // Products come back to back: a look at a barrier waits behind the three products in
                // the queue (200 cycles), so each is issued among the products before the one that
                // needs it, and only what was too early is waited for.
                // tile x of the CTA's own times tile x of the ring, with a look
                auto scores = [&](int x, int32_t i, auto look) {
                    fence_after_sync();
                    const uint64_t p = desc_advance(dA, x * C::TILE), q = desc_advance(dB, ((i & 1) * 2 + x) * C::TILE);
#pragma unroll
                    for (uint32_t s = 0; s < D / 16; ++s) {
                        if (s == D / 32) look();
                        mma_ss(lead, tmem + (x ? TM_DP : TM_S), desc_advance(p, kmajor_off(128, s)),
                               desc_advance(q, kmajor_off(128, s)), id_s, s > 0);
                    }
                    commit_if(lead, x ? &bar.dpfull : &bar.sfull);
                };
                // the weights in tensor memory (rows 0 .. 63 where the first half of the scores
                // was, the others where the second was) times a tile of the ring
                auto gradient = [&](int x, int32_t i, bool more, bool two, auto look) {
                    fence_after_sync();
                    const uint64_t q = desc_advance(dN, ((i & 1) * 2 + (x ^ 1)) * C::TILE);
#pragma unroll
                    for (uint32_t s = 0; s < 8; ++s) {
                        if (s == 4) look();
                        mma_ts(lead, tmem + (x ? TM_DK : TM_DV), tmem + (x ? TM_DP : TM_S) + 8 * (s & 3) + 64 * (s >> 2),
                               desc_advance(q, mnmajor_off(s)), id_d, more || s > 0);
                    }
                    if (two) {
#pragma unroll 1
                        for (uint32_t s = 0; s < 8; ++s)
                            mma_ts(lead, tmem + TM_DK, tmem + TM_DP + 32 + 8 * (s & 3) + 64 * (s >> 2),
                                   desc_advance(q, mnmajor_off(s)), id_d, 1);
                    }
                    // `withhold`: the first tile's dO never leaves its slot (a test hook)
                    commit_if(!more && !x && withhold ? 0u : lead, &bar.empty[x ^ 1][i & 1]);
                };
                bool seen = false;
                auto none = [] {};
                // S of tile i, unless it was the last; a part's last tile: once the rows past its
                // end are zeros
                auto zeroed = [&](int32_t i, int32_t at) {
                    if (at + 1 == per && last < sh.tokens) wait(&bar.statfull[i & 1], (i >> 1) & 1);
                };
                // dP and dV of tile i, S of the next, dK of tile i; `middle`: there are tiles
                // before it, the next one is no part's last, and dS is in one part
                auto turn = [&](auto middle, int32_t i, int32_t next_at, bool two) {
                    constexpr bool kMiddle = decltype(middle)::value;
                    const uint32_t b = i & 1, ph = (i >> 1) & 1, nb = b ^ 1, nph = ((i + 1) >> 1) & 1;
                    const bool next = kMiddle || i + 1 < n, more = kMiddle || i > 0;
                    wait.after(seen, &bar.full[1][b], ph);
                    if (wait.dead()) return;
                    scores(1, i, [&] { seen = mbar_test(&bar.pfull, b); });
                    wait.after(seen, &bar.pfull, b);
                    if (wait.dead()) return;
                    seen = false;
                    gradient(0, i, more, false, [&] { if (next) seen = mbar_test(&bar.full[0][nb], nph); });
                    if (next) {
                        wait.after(seen, &bar.full[0][nb], nph);
                        if (!kMiddle) zeroed(i + 1, next_at);
                        if (wait.dead()) return;
                        scores(0, i + 1, [&] { seen = mbar_test(&bar.dsfull, b); });
                    }
                    wait.after(seen, &bar.dsfull, b);
                    if (wait.dead()) return;
                    gradient(1, i, more, !kMiddle && two, [&] { if (next) seen = mbar_test(&bar.full[1][nb], nph); });
                };
                wait(&bar.afull[0], 0);
                wait(&bar.full[0][0], 0);
                zeroed(0, 0);
                if (!wait.dead()) scores(0, 0, none);
                wait(&bar.afull[1], 0);
                int32_t own = 0, at = per == 1 ? 0 : 1;            // places in their parts: the tile, the next
                for (int32_t i = 0; i < n; ++i) {
                    const bool two = in_two(own);
                    if (i > 0 && i + 1 < n && at + 1 < per && !two) turn(std::true_type(), i, at, two);
                    else turn(std::false_type(), i, at, two);
                    own = at;
                    if (++at == per) at = 0;
                }
                commit_if(lead, &bar.done);                     // no MMA outlives the loop
                mbar_wait(&bar.done, 0);
                __syncwarp();
            }
        } else if (warp == C::WARP_STAT) {
            // -------------------------------------------------------- lse and delta of the rows
            int32_t part = 0, at = 0;
            for (int32_t i = 0; i < n; ++i) {
                const int32_t tokens = at + 1 == per ? last : sh.tokens, b = i & 1;
                const int64_t row0 = (int64_t)(t.seq0 + key0 + at * sh.tokens) * a.Hq +
                                     (hk * sh.parts + part) * sh.heads;
                float l[4], d[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int32_t r = lane + 32 * k, tok = r / sh.heads, g = r - tok * sh.heads;
                    const bool live = tok < tokens;
                    const int64_t x = row0 + (int64_t)tok * a.Hq + g;
                    const float lse = live ? a.lse_in[x] : CUDART_INF_F;
                    // no weight: none to any key
                    l[k] = lse == -CUDART_INF_F ? -CUDART_INF_F : -lse * kAttnLog2e;
                    d[k] = live ? -a.delta[x] : 0.f;
                }
                wait(&bar.statempty[b], ((i >> 1) & 1) ^ 1);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    stats[b * 256 + lane + 32 * k] = l[k];
                    stats[b * 256 + 128 + lane + 32 * k] = d[k];
                }
                if (tokens < sh.tokens) {
                    // rows of the next sequence: zeros, since the gradients add over all rows
                    for (int x = 0; x < 2; ++x) {
                        wait(&bar.full[x][b], (i >> 1) & 1);
                        zero_rows<D>(ring(x, i), tokens * sh.heads, rows, lane, 32);
                    }
                    fence_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.statfull[b]);
                if (++at == per) {
                    at = 0;
                    ++part;
                }
            }
        } else {
            // -------------------------------------------------------- P and dS
            const int half = warp >> 2, key = tid & 127;           // the thread's rows: 64 half ..
            const uint32_t lane0 = tmem_addr(tmem, 32 * (warp & 3), 0);
            const uint32_t s_tm = lane0 + TM_S + 64 * half, dp_tm = lane0 + TM_DP + 64 * half;
            const float2 c = both(a.scale * kAttnLog2e);
            int32_t at = 0;
            for (int32_t i = 0; i < n; ++i) {
                const int32_t b = i & 1;
                const float4* nl = reinterpret_cast<const float4*>(stats + b * 256 + 64 * half);
                const float4* nd = nl + 32;
                // rows before this one are tokens before the key
                const int32_t begin = min(128, max(0, key - at * sh.tokens)) * sh.heads - 64 * half;
                const bool cut = at * sh.tokens < kTcKeys - 1;     // for some key
                const bool two = in_two(at);
                const int32_t used = (at + 1 == per ? last : sh.tokens) * sh.heads - 64 * half;
                if (++at == per) at = 0;
                wait(&bar.statfull[b], (i >> 1) & 1);
                wait(&bar.sfull, i & 1);
                __syncwarp();
                fence_after_sync();
                float p[64];
                tmem_ld32_start(s_tm, p);
                tmem_ld32_start(s_tm + 32, p + 32);
                tmem_ld_wait(p);
                // rows of zeros behind those in use have scores of 0, but NaN with a key that has an infinity
                if (used < 64 && __any_sync(0xffffffffu, p[63] != p[63])) {
#pragma unroll
                    for (int k = 0; k < 64; ++k) p[k] = k < used ? p[k] : 0.f;
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float4 l = nl[k];
                    const float2 x = fma2(make_float2(p[4 * k], p[4 * k + 1]), c, make_float2(l.x, l.y));
                    const float2 y = fma2(make_float2(p[4 * k + 2], p[4 * k + 3]), c, make_float2(l.z, l.w));
                    p[4 * k] = ex2_approx(x.x);
                    p[4 * k + 1] = ex2_approx(x.y);
                    p[4 * k + 2] = ex2_approx(y.x);
                    p[4 * k + 3] = ex2_approx(y.y);
                }
                if (cut) {
#pragma unroll
                    for (int k = 0; k < 64; ++k) p[k] = k < begin ? 0.f : p[k];
                }
                store_pairs(s_tm, p);
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.pfull);
                wait(&bar.dpfull, i & 1);
                __syncwarp();
                fence_after_sync();
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float d[32];
                    tmem_ld32(dp_tm + 32 * x, d);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 e = nd[8 * x + k];
                        float* q = p + 32 * x + 4 * k;
                        const float2 u = mul2(make_float2(q[0], q[1]),
                                              fma2(make_float2(d[4 * k], d[4 * k + 1]), both(1.f), make_float2(e.x, e.y)));
                        const float2 v = mul2(make_float2(q[2], q[3]),
                                              fma2(make_float2(d[4 * k + 2], d[4 * k + 3]), both(1.f), make_float2(e.z, e.w)));
                        q[0] = u.x; q[1] = u.y; q[2] = v.x; q[3] = v.y;
                    }
                }
                if (cut) {
                    // whatever dP is there
#pragma unroll
                    for (int k = 0; k < 64; ++k) p[k] = k < begin ? 0.f : p[k];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.statempty[b]);
                if (two) store_rests(dp_tm, p);
                store_pairs(dp_tm, p);
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.dsfull);
            }
            wait(&bar.done, 0);
            __syncwarp();
            fence_after_sync();
            const int64_t row = ((int64_t)(t.seq0 + key0 + key) * a.Hk + hk) * D;
            store_row<D>(lane0 + (half ? TM_DK : TM_DV), half ? a.scale : 1.f, key < left,
                         static_cast<__nv_bfloat16*>(half ? a.dk : a.dv) + row);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == C::WARP_MMA) {
        fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- dq
template <int D> struct CfgQ {
    static constexpr int HALVES = D / 64;
    static constexpr uint32_t TILE = 128 * D * 2;
    // slots of keys and of values, each in a ring of its own: a tile's keys are held until the
    // product with dS, its values only until dP
    static constexpr int KS = D == 128 ? 3 : 4, VS = D == 128 ? 2 : 4;
    static constexpr uint32_t OFF_K = 2 * TILE, OFF_V = OFF_K + KS * TILE, OFF_BAR = OFF_V + VS * TILE,
                              OFF_SUM = OFF_BAR + 512, SMEM = OFF_SUM + 1024 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
    static constexpr int NT = 352, WARP_LOAD = 8, WARP_MMA = 9, WARP_STORE = 10;
    static constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DQ = 384;      // two buffers of dP
};

struct QBars {
    uint64_t afull[2], aempty[2];      // the rows' queries and dO
    uint64_t kfull[4], kempty[4], vfull[4], vempty[4];         // ring slots
    uint64_t sfull, sempty;
    uint64_t dpfull[2], dsfull[2];     // dP, dS in its place
    uint64_t summed;                   // delta of both halves of the rows' keys
    uint64_t ofull, oempty, staged;    // dq added up, read, in its ring slot
    uint64_t jfull[2], jempty[2];
    uint64_t drain;
    uint32_t tmem;
    int32_t abort;
    AttnJob job[2];
};

template <int D>
__global__ void __launch_bounds__(CfgQ<D>::NT, 1)
attn_bwd_q_tc_kernel(AttnArgs a, AttnShape sh, int32_t jobs, const __grid_constant__ QMaps maps)
{
    using C = CfgQ<D>;
    constexpr int HALVES = C::HALVES, KS = C::KS, VS = C::VS;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    QBars& bar = *reinterpret_cast<QBars*>(sm + C::OFF_BAR);
    static_assert(sizeof(QBars) <= 512, "barriers");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.kfull[i], 1);
            mbar_init(&bar.kempty[i], 1);
            mbar_init(&bar.vfull[i], 1);
            mbar_init(&bar.vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.afull[i], 1);
            mbar_init(&bar.aempty[i], 1);
            mbar_init(&bar.dpfull[i], 1);
            mbar_init(&bar.dsfull[i], 8);
            mbar_init(&bar.jfull[i], 1);
            mbar_init(&bar.jempty[i], 10);
        }
        mbar_init(&bar.sfull, 1);
        mbar_init(&bar.sempty, 8);
        mbar_init(&bar.summed, 8);
        mbar_init(&bar.ofull, 1);
        mbar_init(&bar.oempty, 8);
        mbar_init(&bar.staged, 8);
        mbar_init(&bar.drain, 1);
        bar.abort = 0;
        fence_mbar_init();
        prefetch_map(&maps.q);
        prefetch_map(&maps.dout);
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
    }
    wait_for_previous();
    if (warp == C::WARP_MMA) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = uniform(bar.tmem);
    WarpWait wait(&bar.abort, a.status);

    if (warp == C::WARP_LOAD) {
        // ------------------------------------------------------------ producer
        AttnWalk walk(a, sh.tokens, kTcKeyShift);
        uint32_t ck = 0, cv = 0, loads[2] = {0, 0};
        for (int32_t round = 0; !wait.dead(); ++round) {
            const AttnJob job = attn_job(walk, a, sh, jobs, round);
            wait.for_job(&bar.jempty[round & 1], ((round >> 1) & 1) ^ 1);
            if (wait.dead()) break;            // a role may still read the job that has the place
            if (lane == 0) bar.job[round & 1] = job;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.jfull[round & 1]);
            if (!job.found) break;
            const int32_t n = (attn_keys(a, job.t) + kTcKeys - 1) >> kTcKeyShift, hk = job.unit / sh.parts;
            auto load = [&](unsigned char* dst, const void* map, int y, int z, uint32_t bytes, uint64_t* full) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(full, bytes);
                    for (int h = 0; h < HALVES; ++h) tma_load_3d(dst + h * (128 * 128), map, 64 * h, y, z, full);
                }
                __syncwarp();
            };
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                wait(&bar.aempty[x], (loads[x] & 1) ^ 1);
                if (wait.dead()) continue;
                load(sm + x * C::TILE, x ? &maps.dout : &maps.q, job.unit * sh.heads, job.t.row0,
                     (uint32_t)sh.tokens * sh.heads * 128 * HALVES, &bar.afull[x]);
                ++loads[x];
            }
            for (int32_t i = 0; i < n; ++i) {
                const int32_t key = job.t.seq0 + (i << kTcKeyShift);
                wait(&bar.kempty[ck % KS], ((ck / KS) & 1) ^ 1);
                if (wait.dead()) break;
                load(sm + C::OFF_K + ck % KS * C::TILE, &maps.k, hk, key, C::TILE, &bar.kfull[ck % KS]);
                ++ck;
                wait(&bar.vempty[cv % VS], ((cv / VS) & 1) ^ 1);
                if (wait.dead()) break;
                load(sm + C::OFF_V + cv % VS * C::TILE, &maps.v, hk, key, C::TILE, &bar.vfull[cv % VS]);
                ++cv;
            }
            if (job.t.tokens == sh.tokens) {           // a slot for the gradients
                wait(&bar.vempty[cv % VS], ((cv / VS) & 1) ^ 1);
                if (wait.dead()) break;
                if (lane == 0) mbar_arrive(&bar.vfull[cv % VS]);
                ++cv;
            }
        }
        // every copy has landed before the CTA ends
        if (lane == 0) {
            for (int x = 0; x < 2; ++x)
                if (loads[x] > 0) mbar_wait(&bar.afull[x], (loads[x] - 1) & 1);
            for (uint32_t k = ck > KS ? ck - KS : 0; k < ck; ++k) mbar_wait(&bar.kfull[k % KS], (k / KS) & 1);
            for (uint32_t k = cv > VS ? cv - VS : 0; k < cv; ++k) mbar_wait(&bar.vfull[k % VS], (k / VS) & 1);
        }
        __syncwarp();
    } else if (warp == C::WARP_MMA) {
        // ------------------------------------------------------------ MMA
        constexpr uint32_t id_s = idesc(kFmtBF16, 128, 128), id_d = idesc(kFmtBF16, 128, D, false, true);
        const uint32_t lead = elect_one(), base = smem_u32(sm);
        const uint64_t dA = desc_kmajor(base, 128, 0);
        const uint64_t dK = desc_kmajor(base + C::OFF_K, 128, 0), dV = desc_kmajor(base + C::OFF_V, 128, 0);
        const uint64_t dN = D == 128 ? desc_mnmajor128(base + C::OFF_K, 128 * 128, 0)
                                     : desc_mnmajor64(base + C::OFF_K, 0);
        const bool withhold = a.fault == KDA_TEST_FAULT_ATTENTION_BWD_Q && blockIdx.x == 0;
        uint32_t done = 0;                             // key tiles of the jobs before
        Ring<KS> kr;
        Ring<VS> vr;
        for (int32_t round = 0;; ++round) {
            wait.for_job(&bar.jfull[round & 1], (round >> 1) & 1);
            if (wait.dead()) break;
            const AttnJob& job = bar.job[round & 1];
            if (!uniform(job.found)) break;
            const int32_t all = uniform(attn_keys(a, job.t)), n = (all + kTcKeys - 1) >> kTcKeyShift;
            const int32_t slot = uniform((int32_t)(job.t.tokens == sh.tokens));
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.jempty[round & 1]);
            // Looks at barriers as in the first kernel.  S, then dP, of key tile i:
            auto scores = [&](int x, int32_t i, uint32_t slot, auto look) {
                fence_after_sync();
                const uint32_t b = (done + i) & 1;
                const uint64_t p = desc_advance(dA, x * C::TILE), q = desc_advance(x ? dV : dK, slot * C::TILE);
#pragma unroll
                for (uint32_t s = 0; s < D / 16; ++s) {
                    if (s == D / 32) look();
                    mma_ss(lead, tmem + (x ? C::TM_DP + b * 128 : C::TM_S), desc_advance(p, kmajor_off(128, s)),
                           desc_advance(q, kmajor_off(128, s)), id_s, s > 0);
                }
                commit_if(lead, x ? &bar.dpfull[b] : &bar.sfull);
                if (x) commit_if(lead, &bar.vempty[slot]);
                if (i + 1 == n) commit_if(lead, &bar.aempty[x]);
            };
            bool seen = false;
            // S and dP of tile i + 1, dq of tile i; `middle`: tiles before it and two whole ones behind
            auto turn = [&](auto middle, int32_t i) {
                constexpr bool kMiddle = decltype(middle)::value;
                const uint32_t at = done + i, b = at & 1, k = kr.slot;
                const bool next = kMiddle || i + 1 < n;
                const bool known = seen;
                seen = false;
                if (next) {
                    Ring<KS> kn = kr;
                    kn.next();
                    if (!__all_sync(0xffffffffu, known)) {
                        wait(&bar.kfull[kn.slot], kn.phase);
                        wait(&bar.vfull[vr.slot], vr.phase);
                        wait(&bar.sempty, (at + 1) & 1 ^ 1);
                    }
                    if (wait.dead()) return;
                    scores(0, i + 1, kn.slot, [] {});
                    scores(1, i + 1, vr.slot, [&] { seen = mbar_test(&bar.dsfull[b], (at >> 1) & 1); });
                    vr.next();
                    kr = kn;
                }
                if (!kMiddle && i == 0) wait(&bar.oempty, (round & 1) ^ 1);
                wait.after(seen, &bar.dsfull[b], (at >> 1) & 1);
                if (wait.dead()) return;
                fence_after_sync();
                const uint64_t q = desc_advance(dN, k * C::TILE);
                const int32_t keys = all - (i << kTcKeyShift);
                // dS: keys 0 .. 63 where the first half of dP was, the others where the second was
                auto step = [&](uint32_t s) {
                    mma_ts(lead, tmem + C::TM_DQ, tmem + C::TM_DP + b * 128 + 8 * (s & 3) + 64 * (s >> 2),
                           desc_advance(q, mnmajor_off(s)), id_d, kMiddle || i > 0 || s > 0);
                };
                seen = false;
                if (kMiddle || keys >= kTcKeys) {
#pragma unroll
                    for (uint32_t s = 0; s < 8; ++s) {
                        if (s == 4 && kMiddle) {
                            Ring<KS> kn = kr;
                            kn.next();
                            seen = mbar_test(&bar.kfull[kn.slot], kn.phase) & mbar_test(&bar.vfull[vr.slot], vr.phase) &
                                   mbar_test(&bar.sempty, at & 1 ^ 1);
                        }
                        step(s);
                    }
                } else {
#pragma unroll 1
                    for (uint32_t s = 0; 16 * (int32_t)s < keys; ++s) step(s);
                }
                if (!kMiddle && n == 1) {              // the second parts
#pragma unroll 1
                    for (uint32_t s = 0; 16 * (int32_t)s < keys && s < 8; ++s)
                        mma_ts(lead, tmem + C::TM_DQ, tmem + C::TM_DP + b * 128 + 32 + 8 * (s & 3) + 64 * (s >> 2),
                               desc_advance(q, mnmajor_off(s)), id_d, 1);
                }
                // `withhold`: the first keys never leave their slot (a test hook)
                commit_if(!kMiddle && withhold && i == 0 && round == 0 ? 0u : lead, &bar.kempty[k]);
                if (!kMiddle && i + 1 == n) commit_if(lead, &bar.ofull);
            };
            wait(&bar.afull[0], round & 1);
            wait(&bar.kfull[kr.slot], kr.phase);
            wait(&bar.sempty, (done & 1) ^ 1);
            if (!wait.dead()) scores(0, 0, kr.slot, [] {});
            wait(&bar.afull[1], round & 1);
            wait(&bar.vfull[vr.slot], vr.phase);
            if (!wait.dead()) scores(1, 0, vr.slot, [] {});
            vr.next();
            for (int32_t i = 0; i < n; ++i) {
                if (i > 0 && i + 2 < n) turn(std::true_type(), i);
                else turn(std::false_type(), i);
            }
            kr.next();
            if (slot) vr.next();
            done += n;
        }
        commit_if(lead, &bar.drain);                   // no MMA outlives the loop
        mbar_wait(&bar.drain, 0);
        __syncwarp();
    } else if (warp == C::WARP_STORE) {
        // ------------------------------------------------------------ gradients from their ring slots
        uint32_t cv = 0, count = 0;
        for (int32_t round = 0;; ++round) {
            wait.for_job(&bar.jfull[round & 1], (round >> 1) & 1);
            if (wait.dead()) break;
            const AttnJob job = bar.job[round & 1];
            if (!job.found) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.jempty[round & 1]);
            cv += (attn_keys(a, job.t) + kTcKeys - 1) >> kTcKeyShift;
            if (job.t.tokens != sh.tokens) continue;
            wait.for_job(&bar.staged, count++ & 1);
            if (wait.dead()) break;
            if (lane == 0) {
                for (int h = 0; h < HALVES; ++h)
                    tma_store_3d(&maps.dq, sm + C::OFF_V + cv % VS * C::TILE + h * (128 * 128), 64 * h,
                                 job.unit * sh.heads, job.t.row0);
                tma_store_wait<true>();
                mbar_arrive(&bar.vempty[cv % VS]);
            }
            __syncwarp();
            ++cv;
        }
        if (lane == 0) tma_store_wait<false>();
        __syncwarp();
    } else {
        // ------------------------------------------------------------ P and dS
        const int half = warp >> 2, r = tid & 127;                 // the thread's keys: 64 half ..
        const uint32_t lane0 = tmem_addr(tmem, 32 * (warp & 3), 0);
        const uint32_t s_tm = lane0 + C::TM_S + 64 * half;
        const float2 factor = both(a.scale * kAttnLog2e);
        const int32_t tok = r / sh.heads, g = r - tok * sh.heads;
        float* sums = reinterpret_cast<float*>(sm + C::OFF_SUM);   // [half][row]
        uint32_t cv = 0, done = 0, exact = 0;
        for (int32_t round = 0;; ++round) {
            wait.for_job(&bar.jfull[round & 1], (round >> 1) & 1);
            if (wait.dead()) break;
            const AttnJob job = bar.job[round & 1];
            if (!job.found) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.jempty[round & 1]);
            const AttnTile& t = job.t;
            const int32_t all = attn_keys(a, t), n = (all + kTcKeys - 1) >> kTcKeyShift;
            const bool live = tok < t.tokens;
            const int64_t row = (int64_t)(t.row0 + tok) * a.Hq + job.unit * sh.heads + g;
            const float lse = live ? a.lse_in[row] : CUDART_INF_F;
            const float2 nl = both(lse == -CUDART_INF_F ? -CUDART_INF_F : -lse * kAttnLog2e);
            float2 nd = both(live && n > 1 ? -a.delta[row] : 0.f);
            for (int32_t i = 0; i < n; ++i) {
                // keys from this one on are tokens behind the row's
                const int32_t end = t.pos0 + tok + 1 - (i << kTcKeyShift) - 64 * half;
                const bool cut = ((i + 1) << kTcKeyShift) > t.pos0 + 1;
                const uint32_t at = done + i, b = at & 1, dp_tm = lane0 + C::TM_DP + b * 128 + 64 * half;
                wait(&bar.sfull, at & 1);
                fence_after_sync();
                float p[64];
                tmem_ld32_start(s_tm, p);
                tmem_ld32_start(s_tm + 32, p + 32);
                tmem_ld_wait(p);
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.sempty);
#pragma unroll
                for (int k = 0; k < 64; k += 2) {
                    const float2 x = fma2(make_float2(p[k], p[k + 1]), factor, nl);
                    p[k] = ex2_approx(x.x);
                    p[k + 1] = ex2_approx(x.y);
                }
                wait(&bar.dpfull[b], (at >> 1) & 1);
                fence_after_sync();
                if (n == 1) {
                    // delta from the row's own weights, for the other kernel too
                    float sum = 0.f;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float d[32];
                        tmem_ld32(dp_tm + 32 * x, d);
#pragma unroll
                        for (int k = 0; k < 32; ++k) sum += 32 * x + k < end ? p[32 * x + k] * d[k] : 0.f;
                    }
                    sums[128 * half + r] = sum;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.summed);
                    wait(&bar.summed, exact++ & 1);
                    sum += sums[128 * (half ^ 1) + r];
                    if (half == 0 && live) a.delta[row] = sum;
                    nd = both(-sum);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float d[32];
                    tmem_ld32(dp_tm + 32 * x, d);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float* q = p + 32 * x + k;
                        const float2 u = mul2(make_float2(q[0], q[1]), fma2(make_float2(d[k], d[k + 1]), both(1.f), nd));
                        q[0] = u.x;
                        q[1] = u.y;
                    }
                }
                if (cut) {
#pragma unroll
                    for (int k = 0; k < 64; ++k) p[k] = k < end ? p[k] : 0.f;
                }
                const int32_t keys = all - (i << kTcKeyShift);
                if (keys < kTcKeys && half == 0) {
                    // keys past the end, as far as the product reads (16 at a time); the scores
                    // with them are done
                    zero_rows<D>(sm + C::OFF_K + at % KS * C::TILE, keys, (keys + 15) & ~15, r, 128);
                    fence_async_smem();
                    __syncwarp();
                }
                if (n == 1) store_rests(dp_tm, p);
                store_pairs(dp_tm, p);
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.dsfull[b]);
            }
            wait(&bar.ofull, round & 1);
            fence_after_sync();
            // each half of the warps takes half of the channels
            const uint32_t o_tm = lane0 + C::TM_DQ + D / 2 * half;
            if (t.tokens == sh.tokens) {
                const uint32_t slot = (cv + n) % VS;
                unsigned char* buf = sm + C::OFF_V + slot * C::TILE;
                wait(&bar.vfull[slot], ((cv + n) / VS) & 1);
#pragma unroll
                for (int k = 0; k < D / 2; k += 32) {
                    float x[32];
                    tmem_ld32(o_tm + k, x);
#pragma unroll
                    for (int y = 0; y < 32; y += 8)
                        *reinterpret_cast<uint4*>(buf + sw128_tile(128, r, 2 * (D / 2 * half + k + y))) = make_uint4(
                            pack_bf16(x[y] * a.scale, x[y + 1] * a.scale), pack_bf16(x[y + 2] * a.scale, x[y + 3] * a.scale),
                            pack_bf16(x[y + 4] * a.scale, x[y + 5] * a.scale), pack_bf16(x[y + 6] * a.scale, x[y + 7] * a.scale));
                }
                fence_async_smem();
                ++cv;
            } else {
                store_row<D / 2>(o_tm, a.scale, live, static_cast<__nv_bfloat16*>(a.dq) + row * D + D / 2 * half);
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar.oempty);
                if (t.tokens == sh.tokens) mbar_arrive(&bar.staged);
            }
            cv += n;
            done += n;
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == C::WARP_MMA) {
        fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <int D> cudaError_t backward(const AttnArgs& a, cudaStream_t stream)
{
    using C = Cfg<D>;
    const AttnShape sh = attn_shape(kTcRows, a.Hq, a.Hk);
    KvMaps maps;
    memset(&maps, 0, sizeof(maps));
    cudaError_t e = encode_heads(&maps.q, a.q, a.T, a.Hq, D, a.q_stride, sh.heads, sh.tokens);
    if (e == cudaSuccess) e = encode_heads(&maps.dout, a.dout, a.T, a.Hq, D, (int64_t)a.Hq * D, sh.heads, sh.tokens);
    if (e == cudaSuccess) e = encode_heads(&maps.k, a.k, a.T, a.Hk, D, a.k_stride, 1, kTcKeys);
    if (e == cudaSuccess) e = encode_heads(&maps.v, a.v, a.T, a.Hk, D, a.v_stride, 1, kTcKeys);
    if (e != cudaSuccess) return e;
    QMaps qmaps = {maps.q, maps.dout, maps.k, maps.v, maps.q};
    e = encode_heads(&qmaps.dq, a.dq, a.T, a.Hq, D, (int64_t)a.Hq * D, sh.heads, sh.tokens);
    if (e != cudaSuccess) return e;
    const int64_t kv = attn_items(a.N, a.T, kTcKeys) * a.Hk, q = attn_tiles(a.N, a.T, sh.tokens) * sh.units;
    if (kv > INT32_MAX || q > INT32_MAX) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> set_kv{0}, set_q{0};
    e = allow_smem(attn_bwd_kv_tc_kernel<D>, C::SMEM, &set_kv);
    if (e == cudaSuccess) e = allow_smem(attn_bwd_q_tc_kernel<D>, CfgQ<D>::SMEM, &set_q);
    if (e != cudaSuccess) return e;
    // the first writes delta of some rows for the second
    e = launch_after(attn_bwd_q_tc_kernel<D>, launch_config(q < sm_count() ? q : sm_count(), CfgQ<D>::NT, CfgQ<D>::SMEM),
                     stream, a, sh, (int32_t)q, qmaps);
    if (e != cudaSuccess) return e;
    return launch_after(attn_bwd_kv_tc_kernel<D>, launch_config(kv, C::NT, C::SMEM), stream, a, sh, maps);
}

}  // namespace

cudaError_t launch_attention_bwd_tc(const AttnArgs& a, cudaStream_t stream)
{
    return a.D == 64 ? backward<64>(a, stream) : backward<128>(a, stream);
}

}  // namespace kda
