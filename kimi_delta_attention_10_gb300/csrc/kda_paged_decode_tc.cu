// kda_paged_decode for BF16 caches on the tensor cores (tcgen05).
//
// Per tile of 128 tokens, with the roles of the usual product turned round so that
// the long axis is the MMA's M and the few query heads its N:
//     S[128 tokens, heads]  = K[128, D] Q[heads, D]^T          (M = 128, N = heads)
//     O^T[D, heads]        += V^T[D, 128] P^T[heads, 128]^T    (M = D,   N = 2 heads)
// K and V tiles are read from shared memory exactly as their pages lie in memory
// (K-major keys, MN-major values), so nothing is transposed and nothing padded but
// N.  The weights p = e^(s - m) go back to shared memory as two BF16 rows, the
// rounded value and the rounded rest: N is nearly free here (the MMA's time is the
// 128-row operand's read), and the weights then carry 16 bits instead of 8.  The two rows'
// sums stay apart until they are read: an infinite value is right in the first alone.
//
// HBM-bound: 2 D values a token and key-value head, once.  Warp roles:
//   producers one warp for K, one for V: a TMA box per page and 64 channels into a
//             ring of slots (swizzled as the MMA reads them), the block table read by
//             the lanes;
//   MMA       one thread: S of tile i + 1 is issued before the product with V of
//             tile i, so that it runs while the softmax of tile i does; O adds up in
//             tensor memory over runs of a row's tiles;
//   softmax   four warps per 16 heads, one token a lane.  The reference maximum m
//             moves only when some score of the tile exceeds it by more than 2^8 (p stays
//             within FP32 and BF16 range, the ratios are exact either way): one barrier
//             with a vote per tile, and only after a yes the tile's maxima (a warp
//             reduction, four values through shared memory) and a rescaling of O.
// The CTA's tiles run through all its rows without draining the ring.
//
// Measured (us, and the share of the rate of a plain copy): 64 requests of 0 to 16384
// tokens, 8 key-value heads of 128 channels with 8 query heads each, 302 (98%); two requests
// of 131072 to 262144 256 (98%); 64 of 4096 169 (94%), the tensor pipe 4% busy.  With many
// heads the chain of one tile (scores, vote, weights, product) is longer than its loads and
// nothing runs beside it: 64 requests of 4096 tokens and 4 key-value heads take 95 with groups
// of 16 heads of 128 channels (84%), 98 with 32 (81%), 117 with 64 (69%; 42% of the issue slots,
// the tensor pipe 15%), of 64 channels 57 (69%), 82 (49%) and 103 (39%).  A short row costs about
// 2 us beside its bytes (128 requests of 1 to 600 tokens 46, 48%), one request of 129 tokens 8.6
// with the join.
//
// Tokens past the request's end: their scores are replaced by -infinity, their
// value rows by zeros in shared memory (0 * NaN would not be 0), and pages past the
// end are not loaded.
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

constexpr int kTile = 128;             // tokens per tile
constexpr int kTileShift = 7;
constexpr float kGrowth = 8.f;         // log2 of the growth that moves the reference maximum
// Tiles that O adds up in tensor memory before it joins a total that is rounded: the tensor
// core truncates its sums, so that 262144 values about one lost 1.6e-3 of their mean in one sum.
// Two rows of 131072 to 262144 tokens with FP32 output: 2.5e-5 off in one sum, 5e-6 in runs
// of 32 tiles, in the same time (64 requests of 4096 tokens, groups of 64 heads: 113 -> 117 us
// with runs of 32 tiles, 119 with 16).
constexpr int kRun = 32;

template <int D_, int HP_> struct Cfg {
    static constexpr int D = D_, HP = HP_;             // HP: query heads per unit, padded
    static constexpr int NWG = HP > 16 ? HP / 16 : 1;  // softmax warpgroups: 16 heads of a token a lane
    static constexpr int HW = HP / NWG;                // heads of each
    static constexpr int QR = HP < 16 ? 16 : HP;       // N of the first product
    static constexpr int NPV = 2 * HP;                 // N of the second
    static constexpr int NT = NWG * 128 + 96;
    static constexpr int WARP_K = NWG * 4, WARP_V = WARP_K + 1, WARP_MMA = WARP_K + 2;
    static constexpr int CTAS = D == 64 && HP <= 16 ? 2 : 1;   // per SM
    static constexpr uint32_t SLOT = kTile * D * 2;
    static constexpr uint32_t PBUF = NPV * 256, QBUF = QR * D * 2;
    static constexpr int NQ = HP > 32 ? 1 : 2;         // query buffers
    static constexpr uint32_t MISC = HP <= 8 ? 1024 : HP <= 16 ? 2048 : 80 * HP;   // barriers, maxima, sums
    // shared memory of an SM 228 KB, 1 KB of it kept per CTA; 1 KB for alignment
    // and 1 KB for the static part
    static constexpr uint32_t ROOM = (CTAS == 2 ? 113 * 1024 : 227 * 1024) - 2048;
    static constexpr int NS_ = (ROOM - 2 * PBUF - NQ * QBUF - MISC) / SLOT;
    // 128 KB an SM: with more in flight SMs share the bandwidth less evenly (64 ragged
    // requests 304, 309, 317 us with 4, 5, 6 slots of 32 KB)
    static constexpr int NSMAX = 128 * 1024 / (int)SLOT / CTAS;
    static constexpr int NS = NS_ > NSMAX ? NSMAX : NS_;       // ring slots
    static_assert(NS >= 4, "K and V of two tiles, and no slot in two producers' hands");
    static constexpr uint32_t OFF_P = NS * SLOT, OFF_Q = OFF_P + 2 * PBUF,
                              OFF_MISC = OFF_Q + NQ * QBUF, SMEM = OFF_MISC + MISC + 1024;
    static constexpr uint32_t TM_O = 2 * QR;           // after two S buffers
    static constexpr uint32_t TM_TOTAL = TM_O + NPV, TM_USED = TM_TOTAL + HP;
    static constexpr uint32_t TM_COLS = TM_USED <= 64 ? 64 : TM_USED <= 128 ? 128
                                        : TM_USED <= 256 ? 256 : 512;
    static_assert(TM_COLS * CTAS <= 512, "tensor memory of an SM");
};

struct Maps {
    CUtensorMap q, k, v;
};

struct Bars {
    uint64_t full[8], empty[8];        // ring slots
    uint64_t sfull[2], sempty[2];      // S in tensor memory
    uint64_t pfull[2];                 // P in shared memory
    uint64_t ofull[2];                 // product with V done: O is whole, the P buffer read
    uint64_t qfull[2], qempty[2];
    uint64_t drain;
    uint32_t tmem;
    int32_t abort;
};

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&r)[8])
{
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t a, float (&r)[8]) { tmem_ld8(a, r); }
__device__ __forceinline__ void tmem_ld(uint32_t a, float (&r)[16]) { tmem_ld16(a, r); }

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&r)[8])
{
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(u[0]),
                 "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
                 "r"(taddr)
                 : "memory");
}

// O of the weights' two parts.  An infinite value makes the first infinite (or NaN, as it
// should); times the rest of a weight, which may be zero or negative, it would make NaN.
__device__ __forceinline__ float both_parts(float hi, float lo)
{
    return fabsf(hi) < CUDART_INF_F ? hi + lo : hi;
}

// Sums of N values over the warp's lanes: each step halves the values a lane sums, so that
// l[0] of lane 32 / N * g is the sum of the lanes' l[g].
template <int N, int O = 16, int M>
__device__ __forceinline__ void warp_sums(float (&l)[M], int lane)
{
    if constexpr (N > 1) {
        const bool up = lane & O;
#pragma unroll
        for (int g = 0; g < N / 2; ++g) {
            const float give = up ? l[g] : l[g + N / 2], take = up ? l[g + N / 2] : l[g];
            l[g] = take + __shfl_xor_sync(0xffffffffu, give, O);
        }
    } else {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], O);
    }
    if constexpr (O > 1) warp_sums<(N > 1 ? N / 2 : 1), O / 2>(l, lane);
}

template <int D, int HP>
__global__ void __launch_bounds__(Cfg<D, HP>::NT, Cfg<D, HP>::CTAS)
paged_decode_tc_kernel(DecodeArgs a, DecodeShape sh, const __grid_constant__ Maps maps)
{
    using C = Cfg<D, HP>;
    constexpr int HALVES = D / 64, HW = C::HW, NS = C::NS;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    Bars& bar = *reinterpret_cast<Bars*>(sm + C::OFF_MISC);
    float* s_max = reinterpret_cast<float*>(sm + C::OFF_MISC + 256);     // [2][NWG][4][HW]
    float* s_sum = s_max + 2 * 4 * HP;                                   // [4][HP]
    float* s_inv = s_sum + 4 * HP;                                       // [HP]
    float* s_ref = s_inv + HP;                                           // [4][HP]
    static_assert(sizeof(Bars) <= 256 && 256 + 17 * HP * 4 <= C::MISC, "misc region");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.Hq / a.Hk, groups = sh.units / a.Hk;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.sfull[i], 1);
            mbar_init(&bar.sempty[i], C::NWG * 4);
            mbar_init(&bar.pfull[i], C::NWG * 4);
            mbar_init(&bar.ofull[i], 1);
            mbar_init(&bar.qfull[i], 1);
            mbar_init(&bar.qempty[i], 1);
        }
        mbar_init(&bar.drain, 1);
        bar.abort = 0;
        fence_mbar_init();
    }
    // Tensor memory after the wait: a kernel that lets this one start early may still have
    // its own to allocate, and would never end if this one held it.
    wait_for_previous();
    if (warp == C::WARP_MMA) {
        tmem_alloc(&bar.tmem, C::TM_COLS);
        tmem_relinquish();
    }
    DecodeLens lens;
    lens.load(a);
    fence_before_sync();
    __syncthreads();                               // the barriers and the tensor memory
    fence_after_sync();
    char* ws = static_cast<char*>(a.workspace);
    const DecodeRange rg = decode_range<C::NT>(a, sh, lens, ws);
    const uint32_t tmem = bar.tmem;

    BoundedWait wait(&bar.abort, a.status);
    DecodeWalk w(rg, a, sh, groups);
    if (warp == C::WARP_K || warp == C::WARP_V) {
        // ------------------------------------------------------------ producers
        const bool keys = warp == C::WARP_K;
        const void* map = keys ? &maps.k : &maps.v;
        const int row_shift = a.page_shift < kTileShift ? a.page_shift : kTileShift;
        const int rows = 1 << row_shift;                           // tokens per box
        uint32_t i = 0, item = 0;                                  // tiles and rows so far
        const int half = lane % HALVES, token = lane / HALVES << row_shift;
        int t = 0;
        DecodeTile tile;
        bool more = tile.next(w, t, a, sh, kTile, row_shift, token);
        for (; more; ++i, more = tile.next(w, t, a, sh, kTile, row_shift, token)) {
            if (keys && tile.opens) {
                const uint32_t qb = item % C::NQ;
                wait(&bar.qempty[qb], ((item / C::NQ) & 1) ^ 1);
                wait.dead = __any_sync(0xffffffffu, wait.dead);
                if (wait.dead) break;
                if (lane == 0) mbar_arrive_expect_tx(&bar.qfull[qb], C::QBUF);
                __syncwarp();
                if (lane < HALVES)
                    tma_load_2d(smem_u32(sm + C::OFF_Q + qb * C::QBUF + lane * C::QR * 128),
                                &maps.q, 64 * lane, tile.n * a.Hq + tile.hk * G + tile.part * HP,
                                &bar.qfull[qb]);
                ++item;
            }
            const uint32_t c = 2 * i + (keys ? 0 : 1), slot = c % NS;
            wait(&bar.empty[slot], ((c / NS) & 1) ^ 1);
            wait.dead = __any_sync(0xffffffffu, wait.dead);
            if (wait.dead) break;
            if (lane == 0) mbar_arrive_expect_tx(&bar.full[slot], tile.boxes * HALVES * rows * 128);
            __syncwarp();
            if (lane < tile.boxes * HALVES)
                tma_load_2d(smem_u32(sm + slot * C::SLOT + half * (kTile * 128) + token * 128), map,
                            64 * half, page_row(a, tile.entry, tile.hk, tile.at), &bar.full[slot]);
        }
        // every copy has landed before the CTA ends (all were waited for, unless a wait gave up)
        if (lane == 0) {
            for (uint32_t k = i > (uint32_t)NS ? i - NS : 0; k < i; ++k) {
                const uint32_t c = 2 * k + (keys ? 0 : 1);
                if (c + NS >= 2 * i) mbar_wait(&bar.full[c % NS], (c / NS) & 1);
            }
            for (uint32_t k = item > (uint32_t)C::NQ ? item - C::NQ : 0; k < item; ++k)
                mbar_wait(&bar.qfull[k % C::NQ], (k / C::NQ) & 1);
        }
    } else if (warp == C::WARP_MMA) {
        // ------------------------------------------------------------ MMA
        if (lane == 0) {
            constexpr uint32_t id_s = idesc(kFmtBF16, kTile, C::QR);
            constexpr uint32_t id_o = idesc(kFmtBF16, D, C::NPV, true, false);
            const uint64_t dK = desc_kmajor(smem_u32(sm), kTile, 0);
            const uint64_t dV = D == 128 ? desc_mnmajor128(smem_u32(sm), kTile * 128, 0)
                                         : desc_mnmajor64(smem_u32(sm), 0);
            const uint64_t dQ = desc_kmajor(smem_u32(sm + C::OFF_Q), C::QR, 0);
            const uint64_t dP = desc_kmajor(smem_u32(sm + C::OFF_P), C::NPV, 0);
            uint32_t i = 0, item = 0;
            // the product with V that tile i - 1 still needs: its tokens, and whether it is
            // its row's first here
            int tokens = 0;
            bool begins = false;
            auto product_with_v = [&] {
                const uint32_t t = i - 1, slot = (2 * t + 1) % NS, b = t & 1;
                wait(&bar.full[slot], ((2 * t + 1) / NS) & 1);
                wait(&bar.pfull[b], (t >> 1) & 1);
                if (!wait.dead) {
                    fence_after_sync();
                    auto step = [&](int s) {
                        mma_bf16(tmem + C::TM_O, desc_advance(dV, slot * C::SLOT + mnmajor_off(s)),
                                 desc_advance(dP, b * C::PBUF + kmajor_off(C::NPV, s)), id_o,
                                 s > 0 || !begins);
                    };
                    if (tokens >= kTile) {
#pragma unroll
                        for (int s = 0; s < kTile / 16; ++s) step(s);
                    } else {
                        for (int s = 0; 16 * s < tokens; ++s) step(s);
                    }
                    commit(&bar.empty[slot]);
                    commit(&bar.ofull[b]);
                }
                tokens = 0;
            };
            while (w.next(a, sh)) {
                const uint32_t qb = item % C::NQ, q_phase = (item / C::NQ) & 1;
                for (int t = w.tile0; t < w.tile1; ++t) {
                    const uint32_t slot = (2 * i) % NS, b = i & 1;
                    const uint32_t k_phase = ((2 * i) / NS) & 1, s_phase = ((i >> 1) & 1) ^ 1;
                    // Between rows: the new row's scores go first where they can at once, and
                    // run beside the old row's softmax; else the old row is not kept waiting.
                    if (t == w.tile0 && tokens &&
                        !(mbar_test(&bar.qfull[qb], q_phase) && mbar_test(&bar.full[slot], k_phase) &&
                          mbar_test(&bar.sempty[b], s_phase)))
                        product_with_v();
                    if (t == w.tile0) wait(&bar.qfull[qb], q_phase);
                    wait(&bar.full[slot], k_phase);
                    wait(&bar.sempty[b], s_phase);
                    if (!wait.dead) {
                        fence_after_sync();
#pragma unroll
                        for (int s = 0; s < D / 16; ++s)
                            mma_bf16(tmem + b * C::QR,
                                     desc_advance(dK, slot * C::SLOT + kmajor_off(kTile, s)),
                                     desc_advance(dQ, qb * C::QBUF + kmajor_off(C::QR, s)), id_s,
                                     s > 0);
                        commit(&bar.empty[slot]);
                        if (t + 1 == w.tile1) commit(&bar.qempty[qb]);
                        commit(&bar.sfull[b]);
                    }
                    if (tokens) product_with_v();
                    begins = ((t - w.tile0) & (kRun - 1)) == 0;
                    tokens = w.L - (t << kTileShift);      // more than a tile's: a whole one
                    ++i;
                }
                ++item;
            }
            if (tokens) product_with_v();
            commit(&bar.drain);                            // no MMA outlives the loop
            mbar_wait(&bar.drain, 0);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int wg = warp >> 2, quad = warp & 3, row = tid & 127;     // row: token, then channel
        const uint32_t tlane = tmem_addr(tmem, 32 * quad, 0);
        const float c = a.scale * kLog2e;
        const int bar_id = 1 + wg;
        // the row's place in a P row: 128-byte rows of 64 tokens
        const uint32_t p_base = smem_u32(sm + C::OFF_P) + (row >> 6) * (C::NPV * 128) +
                                (row & 7) * 2 + wg * HW * 128;
        const uint32_t p_chunk = (row >> 3) & 7;
        float2* ws_ml = reinterpret_cast<float2*>(ws + decode_ml_offset(sh));
        float* ws_o = reinterpret_cast<float*>(ws + decode_o_offset(sh));
        float* my_ref = s_ref + quad * HP + wg * HW;       // the warp's copy
        uint32_t i = 0;
        while (w.next(a, sh)) {
            float ref[HW], l[HW];
#pragma unroll
            for (int g = 0; g < HW; ++g) {
                ref[g] = -CUDART_INF_F;
                l[g] = 0.f;
            }
            bool open = true;                              // some reference is still -infinity
            // O's heads g0 .. g0 + 7 in x; the total's added to it, from its references to these
            auto sum8 = [&](int g0, float (&x)[8]) {
                float y[8];
                tmem_ld8(tlane + C::TM_O + wg * HW + g0, x);
                tmem_ld8(tlane + C::TM_O + HP + wg * HW + g0, y);
#pragma unroll
                for (int g = 0; g < 8; ++g) x[g] = both_parts(x[g], y[g]);
            };
            auto add_total = [&](int g0, float (&x)[8]) {
                float y[8];
                tmem_ld8(tlane + C::TM_TOTAL + wg * HW + g0, y);
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const float m = ref[g0 + g], old = my_ref[g0 + g];
                    x[g] = fmaf(y[g], old == m ? 1.f : exp2f(old - m), x[g]);
                }
            };
            for (int t0 = w.tile0;;) {
                const int t1 = min(t0 + kRun, w.tile1);
                for (int t = t0; t < t1; ++t, ++i) {
                    const uint32_t b = i & 1;
                    const int valid = w.L - (t << kTileShift);
                    float s[HW];
                    wait(&bar.sfull[b], (i >> 1) & 1);
                    __syncwarp();
                    fence_after_sync();
                    tmem_ld(tlane + b * C::QR + wg * HW, s);
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.sempty[b]);
                    if (valid < kTile) {
#pragma unroll
                        for (int g = 0; g < HW; ++g) s[g] = row < valid ? s[g] * c : -CUDART_INF_F;
                    } else {
#pragma unroll
                        for (int g = 0; g < HW; ++g) s[g] *= c;
                    }
                    bool grown = open;                     // uniform over the warpgroup
                    if (!grown) {
                        float over = -CUDART_INF_F;
#pragma unroll
                        for (int g = 0; g < HW; ++g) over = fmaxf(over, s[g] - ref[g]);
                        grown = named_sync_or(bar_id, 128, over > kGrowth);
                    }
                    if (grown) {
                        float* maxima = s_max + (b * C::NWG + wg) * 4 * HW;
                        float mine = 0.f;
#pragma unroll
                        for (int g = 0; g < HW; ++g) {
                            const float m = warp_max(s[g]);
                            if (lane == g) mine = m;
                        }
                        if (lane < HW) maxima[quad * HW + lane] = mine;
                        if (t > t0) wait(&bar.ofull[b ^ 1], ((i - 1) >> 1) & 1);
                        named_sync(bar_id, 128);
                        open = false;
#pragma unroll
                        for (int g0 = 0; g0 < HW; g0 += 8) {
                            float keep[8];
                            bool moved = false;
#pragma unroll
                            for (int g = 0; g < 8; ++g) {
                                const float* x = maxima + g0 + g;
                                const float top = fmaxf(fmaxf(x[0], x[HW]), fmaxf(x[2 * HW], x[3 * HW]));
                                keep[g] = 1.f;
                                if (top > ref[g0 + g] + kGrowth) {
                                    keep[g] = exp2f(ref[g0 + g] - top);
                                    ref[g0 + g] = top;
                                    l[g0 + g] *= keep[g];
                                    moved = true;
                                }
                                open |= ref[g0 + g] == -CUDART_INF_F;
                            }
                            if (t > t0 && moved) {
                                fence_after_sync();
#pragma unroll
                                for (int part = 0; part < 2; ++part) {
                                    const uint32_t o = tlane + C::TM_O + part * HP + wg * HW + g0;
                                    float x[8];
                                    tmem_ld8(o, x);
#pragma unroll
                                    for (int g = 0; g < 8; ++g) x[g] *= keep[g];
                                    tmem_st8(o, x);
                                }
                                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                            }
                        }
                    }
                    // the P buffer's last reader
                    if (i >= 2) wait(&bar.ofull[b], ((i - 2) >> 1) & 1);
                    const uint32_t p = p_base + b * C::PBUF;
#pragma unroll
                    for (int g = 0; g < HW; g += 2) {
                        float e[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            // all scores so far -infinity: nothing to subtract
                            const float m = ref[g + k] == -CUDART_INF_F ? 0.f : ref[g + k];
                            e[k] = ex2_approx(s[g + k] - m);
                            l[g + k] += e[k];
                        }
                        const uint32_t hi = pack_bf16(e[0], e[1]);
                        const uint32_t lo = pack_bf16(e[0] - __uint_as_float(hi << 16),
                                                      e[1] - __uint_as_float(hi & 0xffff0000u));
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            // row g + k of the warpgroup's (HW and HP are multiples of 8)
                            const uint32_t at = p + ((g + k) >> 3) * 1024 + ((g + k) & 7) * 128 +
                                                ((p_chunk ^ ((g + k) & 7)) << 4);
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at),
                                         "h"((uint16_t)(k ? hi >> 16 : hi & 0xffffu)) : "memory");
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + HP * 128),
                                         "h"((uint16_t)(k ? lo >> 16 : lo & 0xffffu)) : "memory");
                        }
                    }
                    if (valid < kTile && wg == 0) {
                        // value rows past the end, once they have landed
                        const uint32_t slot = (2 * i + 1) % NS;
                        wait(&bar.full[slot], ((2 * i + 1) / NS) & 1);
                        // as far as the product reads: its steps are 16 tokens
                        const int rows = ((valid + 15) & ~15) - valid;
                        for (int e = row; e < rows * 8 * HALVES; e += 128)
                            *reinterpret_cast<uint4*>(sm + slot * C::SLOT + ((e >> 3) % HALVES) * (kTile * 128) +
                                                      (valid + (e >> 3) / HALVES) * 128 + (e & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.pfull[b]);
                }
                // the run's last product; the next one overwrites O after the next pfull
                wait(&bar.ofull[(i - 1) & 1], ((i - 1) >> 1) & 1);
                __syncwarp();
                fence_after_sync();
                if (__builtin_expect(t1 == w.tile1, 1)) break;
#pragma unroll
                for (int g0 = 0; g0 < HW; g0 += 8) {
                    float x[8];
                    sum8(g0, x);
                    if (t0 > w.tile0) add_total(g0, x);
                    tmem_st8(tlane + C::TM_TOTAL + wg * HW + g0, x);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int g = 0; g < HW; ++g) my_ref[g] = ref[g];
                }
                __syncwarp();
                t0 = t1;
            }
            float acc[HW];
            tmem_ld(tlane + C::TM_O + wg * HW, acc);
            {
                float x[HW];
                tmem_ld(tlane + C::TM_O + HP + wg * HW, x);
#pragma unroll
                for (int g = 0; g < HW; ++g) acc[g] = both_parts(acc[g], x[g]);
            }
            if (__builtin_expect(w.tile1 - w.tile0 > kRun, 0)) {
#pragma unroll
                for (int g0 = 0; g0 < HW; g0 += 8) {
                    float x[8];
#pragma unroll
                    for (int g = 0; g < 8; ++g) x[g] = acc[g0 + g];
                    add_total(g0, x);
#pragma unroll
                    for (int g = 0; g < 8; ++g) acc[g0 + g] = x[g];
                }
            }
            warp_sums<HW>(l, lane);
            constexpr int EACH = 32 / HW;
            if (lane % EACH == 0) s_sum[quad * HP + wg * HW + lane / EACH] = l[0];
            named_sync(bar_id, 128);
            const int hk = w.hk, g0 = w.part * HP + wg * HW;
            const bool whole = w.tile0 == 0 && w.tile1 == w.tiles;
            const int64_t r0 = whole ? (int64_t)w.n * a.Hq + hk * G + g0
                                     : (2 * (int64_t)blockIdx.x + (w.tile0 == 0)) * HP + wg * HW;
            const int heads = min(HW, G - g0);
            // thread g finishes head g's statistics
            float inv = 0.f;
            if (row < heads) {
                const float* sp = s_sum + wg * HW + row;
                const float sum = sp[0] + sp[HP] + sp[2 * HP] + sp[3 * HP];
                float m = ref[0];
#pragma unroll
                for (int g = 1; g < HW; ++g) m = row == g ? ref[g] : m;
                if (!whole)
                    ws_ml[r0 + row] = make_float2(m, sum);
                else if (a.lse != nullptr)
                    a.lse[r0 + row] = m * kLn2 + logf(sum);
                inv = whole ? 1.f / sum : 1.f;
                s_inv[wg * HW + row] = inv;
            }
            named_sync(bar_id, 128);
            // D = 64: a warp's tensor-memory lanes 0 .. 15 hold channels 16 quad ..
            const int ch = D == 128 ? row : 16 * quad + lane;
            const bool mine = D == 128 || lane < 16;
            if (whole && a.out_bf16) {
                __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.out) + r0 * D + ch;
#pragma unroll
                for (int g = 0; g < HW; ++g)
                    if (mine && g < heads) store_one(y + g * D, acc[g] * s_inv[wg * HW + g]);
            } else {
                float* y = (whole ? static_cast<float*>(a.out) : ws_o) + r0 * D + ch;
#pragma unroll
                for (int g = 0; g < HW; ++g)
                    if (mine && g < heads) y[g * D] = acc[g] * s_inv[wg * HW + g];
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == C::WARP_MMA) {
        fence_after_sync();
        tmem_dealloc(tmem, C::TM_COLS);
    }
}

// ---------------------------------------------------------------- launch
int padded_heads(int G)
{
    return G <= 8 ? 8 : G <= 16 ? 16 : G <= 32 ? 32 : 64;
}

template <int D, int HP>
cudaError_t launch_typed(const DecodeArgs& a, const DecodeShape& s, cudaStream_t stream)
{
    using C = Cfg<D, HP>;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    const int page = 1 << a.page_shift;
    const int64_t rows = (int64_t)a.num_pages * a.Hk * page;
    const int64_t qrows = (int64_t)a.N * a.Hq;
    const int box = page < kTile ? page : kTile;
    cudaError_t e = encode_rows(&maps.q, a.q, true, qrows, D, 64, C::QR, true);
    // an empty cache has no page to read: the maps only have to be valid
    if (e == cudaSuccess) e = encode_rows(&maps.k, rows ? a.k : a.q, true, rows ? rows : qrows, D, 64, box, true);
    if (e == cudaSuccess) e = encode_rows(&maps.v, rows ? a.v : a.q, true, rows ? rows : qrows, D, 64, box, true);
    if (e != cudaSuccess) return e;
    auto kern = paged_decode_tc_kernel<D, HP>;
    static std::atomic<uint64_t> set{0};
    e = allow_smem(kern, C::SMEM, &set);
    if (e != cudaSuccess) return e;
    return launch_after(kern, launch_config(s.ctas, C::NT, C::SMEM), stream, a, s, maps);
}

}  // namespace

DecodeShape decode_tc_shape(const DecodeArgs& a)
{
    const int G = a.Hq / a.Hk, hp = padded_heads(G);
    DecodeShape s;
    s.heads = hp;
    s.units = a.Hk * ((G + hp - 1) / hp);
    s.ctas = sm_count() * (a.D == 64 && hp <= 16 ? 2 : 1);
    s.tile_shift = kTileShift;
    s.start = 1;
    return s;
}

cudaError_t launch_paged_decode_tc(const DecodeArgs& a, const DecodeShape& s, cudaStream_t stream)
{
    if (a.D == 64) {
        switch (s.heads) {
            case 8: return launch_typed<64, 8>(a, s, stream);
            case 16: return launch_typed<64, 16>(a, s, stream);
            case 32: return launch_typed<64, 32>(a, s, stream);
            default: return launch_typed<64, 64>(a, s, stream);
        }
    }
    switch (s.heads) {
        case 8: return launch_typed<128, 8>(a, s, stream);
        case 16: return launch_typed<128, 16>(a, s, stream);
        case 32: return launch_typed<128, 32>(a, s, stream);
        default: return launch_typed<128, 64>(a, s, stream);
    }
}

}  // namespace kda
