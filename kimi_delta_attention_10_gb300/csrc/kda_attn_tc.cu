// Attention for several tokens a sequence, BF16 on the tensor cores (tcgen05): the forward
// over packed or paged keys.
//
// A CTA walks over jobs: two tiles of 128 rows (tokens times the heads of a group) that
// share the stream of their key tiles, or a piece of it.  Per tile of 128 keys and each of the two
//     S[128, 128]  = Q[128, D] K[128, D]^T      both operands in shared memory
//     O[128, D]   += P[128, 128] V[128, D]      P in tensor memory, where S was
// so that one tile's softmax runs while the tensor core works for the other.  Warp roles:
//   softmax   four warps a tile, one row a thread: no reduction crosses a thread.  The
//             reference maximum m moves only when it would grow by more than 2^8 (exact
//             either way), and then the thread's warp rescales O in tensor memory; the weights
//             e^(s - m) are rounded to BF16 (2^-8 each; their sum adds them up unrounded);
//   producer  one warp: the walk over the jobs, then K and V tiles through a ring of slots by
//             TMA, a box of 64 channels, or of a page's tokens of them, at a time, and Q;
//   MMA       one warp.  S of the next key tile is issued behind the product with V that reads
//             P in its place.  It has the tensor pipe's time to itself, so what lies between
//             its products is what the kernel loses: operands that the compiler does not know
//             to be uniform, looks at barriers, conditions (5.6 ms at first for 16384 tokens);
//   store     two warps: outputs leave through ring slots by TMA.
//
// Bound by the tensor pipe in long sequences, and there by power: 16384 tokens, 64 / 8 heads of 128
// channels, 2.8 ms, 1570 TFLOP/s, 83% of what a library product reaches in a burst and 94% of what
// it holds.  Pieces of prompts (16 requests, up to 512 tokens over up to 16384) 0.79 ms, 1410
// TFLOP/s.  With few rows by HBM: 64 requests of 4 drafted tokens over up to 16384, 322 us, 93% of
// the rate of a plain copy.  Short sequences by a job's start and end: a job of one tile of rows and
// one of keys takes 7.4 us (64 channels) or 8.9 (128), of two and two 12 or 14.6, a further tile of
// keys about one; 8 sequences of 1 to 2048 tokens 187 us, 860 TFLOP/s; 129 tokens 8.7 us.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "kda_attn_tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr float kGrowth = 8.f;                 // log2 of the growth that moves the reference

constexpr uint32_t kMisc = 640;                // bytes for barriers and jobs

template <int D> struct Cfg {
    static constexpr int HALVES = D / 64;
    static constexpr uint32_t QTILE = kTcRows * D * 2, SLOT = kTcKeys * D * 2;
    static constexpr int NS = D == 128 ? 5 : 8;                // ring slots: 160, 128 KB
    static constexpr uint32_t OFF_KV = 2 * QTILE, OFF_BAR = OFF_KV + NS * SLOT, SMEM = OFF_BAR + kMisc + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
    static constexpr int NT = 384, WARP_LOAD = 8, WARP_MMA = 9, WARP_STORE = 10;   // and 11
    // registers of a thread: at launch, then of the softmax's threads, of the others
    static constexpr int REGS = 168, REGS_SOFTMAX = 208, REGS_OTHER = 88;
    static_assert(2 * REGS_SOFTMAX + REGS_OTHER <= 3 * REGS, "registers of the block");
    static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
};

struct Maps {
    CUtensorMap q, k, v, out;
};

// What a job is for each of its two tiles of rows; worked out once, by the warp that finds it.
struct Plan {
    int32_t tokens[2], keys[2];        // tokens, and keys that its last token sees
    int32_t n[2], steps;               // key tiles in this piece, and the most of them
    int32_t all, j0;                   // keys that any row sees, first key tile
    int32_t slot[2];                   // 1: the rows leave through a ring slot
    __device__ __forceinline__ void set(const AttnArgs& a, const AttnShape& sh, const AttnJob& job)
    {
        const AttnTile& t = job.t;
        tokens[0] = min(t.tokens, sh.tokens);
        tokens[1] = t.tokens - tokens[0];
        all = attn_keys(a, t);
        const int32_t tiles = (int32_t)(((int64_t)all + kTcKeys - 1) >> kTcKeyShift);
        int32_t j1 = tiles;
        j0 = 0;
        if (a.splits > 1) {                // the quotients are a microsecond of a short call
            j0 = (int32_t)((int64_t)tiles * job.piece / a.splits);
            j1 = (int32_t)((int64_t)tiles * (job.piece + 1) / a.splits);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            keys[m] = tokens[m] == 0 ? 0
                      : a.causal     ? max(0, t.pos0 + m * sh.tokens + tokens[m])
                                     : t.kv_len;
            n[m] = max(0, min(j1, (int32_t)(((int64_t)keys[m] + kTcKeys - 1) >> kTcKeyShift)) - j0);
            slot[m] = n[m] > 0 && tokens[m] == sh.tokens && a.pieces == 1;
        }
        steps = max(n[0], n[1]);
    }
};
struct Job : AttnJob {
    Plan p;
};

struct Bars {
    uint64_t full[8], empty[8];        // ring slots
    uint64_t qfull[2], qempty[2];
    uint64_t sfull[2];                 // S in tensor memory
    uint64_t pfull[2];                 // P in its place
    uint64_t ofull[2];                 // product with V done
    uint64_t oempty[2];                // O read
    uint64_t staged[2];                // and in its ring slot
    uint64_t jfull[2], jempty[2];
    uint64_t drain;
    uint32_t tmem;
    int32_t abort;
    Job job[2];
};

// The D values of a thread's row of O, scaled, to the output or a piece of it.
template <int D>
__device__ __forceinline__ void store_row(uint32_t o_tmem, float inv, bool live, __nv_bfloat16* out, float* piece)
{
#pragma unroll
    for (int c = 0; c < D; c += 32) {
        float x[32];
        __syncwarp();
        tmem_ld32(o_tmem + c, x);
        if (!live) {
        } else if (piece != nullptr) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(piece + c + i) =
                    make_float4(x[i] * inv, x[i + 1] * inv, x[i + 2] * inv, x[i + 3] * inv);
        } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
                *reinterpret_cast<uint4*>(out + c + i) = make_uint4(
                    pack_bf16(x[i] * inv, x[i + 1] * inv), pack_bf16(x[i + 2] * inv, x[i + 3] * inv),
                    pack_bf16(x[i + 4] * inv, x[i + 5] * inv), pack_bf16(x[i + 6] * inv, x[i + 7] * inv));
        }
    }
    __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::NT, 1)
attn_fwd_tc_kernel(AttnArgs a, AttnShape sh, int32_t jobs, const __grid_constant__ Maps maps)
{
    using C = Cfg<D>;
    constexpr int HALVES = C::HALVES, NS = C::NS;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    Bars& bar = *reinterpret_cast<Bars*>(sm + C::OFF_BAR);
    static_assert(sizeof(Bars) <= kMisc, "barriers");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.qfull[i], 1);
            mbar_init(&bar.qempty[i], 1);
            mbar_init(&bar.sfull[i], 1);
            mbar_init(&bar.pfull[i], 4);
            mbar_init(&bar.ofull[i], 1);
            mbar_init(&bar.oempty[i], 4);
            mbar_init(&bar.staged[i], 4);
            mbar_init(&bar.jfull[i], 1);
            mbar_init(&bar.jempty[i], 11);
        }
        mbar_init(&bar.drain, 1);
        bar.abort = 0;
        fence_mbar_init();
        prefetch_map(&maps.q);
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
        prefetch_map(&maps.out);
    }
    wait_for_previous();
    if (warp == C::WARP_MMA) {
        tmem_alloc(&bar.tmem, C::TM_COLS);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = uniform(bar.tmem);
    WarpWait wait(&bar.abort, a.status);

    if (warp >= 8) {
        fewer_registers<C::REGS_OTHER>();
        if (warp == C::WARP_LOAD) {
            // -------------------------------------------------------- producer
            AttnWalk walk(a, 2 * sh.tokens, kTcKeyShift);
            if (blockIdx.x == 0 && lane == 0 && a.pieces > 1)
                *static_cast<int32_t*>(a.workspace) = walk.bad ? 0 : a.cu[a.N];
            // a box: rows of a page, or a whole tile; the lane's part of a tile
            const int shift = a.table == nullptr || a.page_shift > kTcKeyShift ? kTcKeyShift : a.page_shift;
            const int half = lane % HALVES, token = lane / HALVES << shift;
            const bool mine = lane / HALVES < kTcKeys >> shift;
            const uint32_t qbytes = (uint32_t)sh.tokens * sh.heads * 128 * HALVES;
            uint32_t c = 0, loads[2] = {0, 0};
            // the first queries wait as if their place were never given back (a test hook)
            const uint32_t lost = a.fault == KDA_TEST_FAULT_ATTENTION && blockIdx.x == 0;
            for (int32_t round = 0; !wait.dead(); ++round) {
                Job job;
                static_cast<AttnJob&>(job) = attn_job(walk, a, sh, jobs, round);
                if (job.found) job.p.set(a, sh, job);
                const Plan& p = job.p;
                wait.for_job(&bar.jempty[round & 1], ((round >> 1) & 1) ^ 1);
                if (wait.dead()) break;        // a role may still read the job that has the place
                if (lane == 0) bar.job[round & 1] = job;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.jfull[round & 1]);
                if (!job.found) break;
                const int32_t hk = job.unit / sh.parts;
                auto load_q = [&](int m) {
                    if (p.n[m] == 0) return;
                    wait(&bar.qempty[m], (loads[m] & 1) ^ 1 ^ lost);
                    if (wait.dead()) return;
                    if (lane == 0) mbar_arrive_expect_tx(&bar.qfull[m], qbytes);
                    __syncwarp();
                    if (lane < HALVES)
                        tma_load_3d(sm + m * C::QTILE + lane * (kTcRows * 128), &maps.q, 64 * lane,
                                    job.unit * sh.heads, job.t.row0 + m * sh.tokens, &bar.qfull[m]);
                    ++loads[m];
                };
                int32_t row = 0;
                auto find_row = [&](int32_t j) {
                    const int32_t k = (j << kTcKeyShift) + token;
                    if (a.table != nullptr && mine && k < p.all) row = (int32_t)attn_page_row(a, job.t.n, hk, k);
                };
                if (p.steps > 0) find_row(p.j0);
                for (int32_t i = 0; i < p.steps && !wait.dead(); ++i) {
                    const int32_t j = p.j0 + i, left = p.all - (j << kTcKeyShift);
                    const int32_t boxes = (min(left, kTcKeys) + (1 << shift) - 1) >> shift;
                    const int32_t here = row;
                    if (i + 1 < p.steps) find_row(j + 1);
                    for (int kv = 0; kv < 2; ++kv, ++c) {
                        const uint32_t slot = c % NS;
                        wait(&bar.empty[slot], ((c / NS) & 1) ^ 1);
                        if (wait.dead()) break;
                        if (lane == 0)
                            mbar_arrive_expect_tx(&bar.full[slot], (uint32_t)(boxes * HALVES) << (shift + 7));
                        __syncwarp();
                        if (lane < boxes * HALVES) {
                            unsigned char* dst = sm + C::OFF_KV + slot * C::SLOT + half * (kTcKeys * 128) + token * 128;
                            const void* map = kv ? &maps.v : &maps.k;
                            if (a.table != nullptr)
                                tma_load_2d(smem_u32(dst), map, 64 * half, here, &bar.full[slot]);
                            else
                                tma_load_3d(dst, map, 64 * half, hk, job.t.seq0 + (j << kTcKeyShift), &bar.full[slot]);
                        }
                    }
                    if (i == 0) {              // their places may still be the last job's
                        load_q(0);
                        load_q(1);
                    }
                }
                // slots for the outputs
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (!p.slot[m] || wait.dead()) continue;
                    wait(&bar.empty[c % NS], ((c / NS) & 1) ^ 1);
                    if (wait.dead()) continue;
                    if (lane == 0) mbar_arrive(&bar.full[c % NS]);
                    ++c;
                }
            }
            // every copy has landed before the CTA ends
            if (lane == 0) {
                for (int m = 0; m < 2; ++m)
                    if (loads[m] > 0) mbar_wait(&bar.qfull[m], (loads[m] - 1) & 1);
                for (uint32_t k = c > (uint32_t)NS ? c - NS : 0; k < c; ++k)
                    mbar_wait(&bar.full[k % NS], (k / NS) & 1);
            }
            __syncwarp();
        } else if (warp == C::WARP_MMA) {
            // -------------------------------------------------------- MMA
            // a negative scale's sign goes into the products, so that their order is the scores'
            const uint32_t id_s = idesc(kFmtBF16, kTcRows, kTcKeys) | (a.scale < 0.f ? kNegateA : 0u);
            constexpr uint32_t id_o = idesc(kFmtBF16, kTcRows, D, false, true);
            const uint32_t lead = elect_one();
            const uint64_t dQ = desc_kmajor(smem_u32(sm), kTcRows, 0);
            const uint64_t dK = desc_kmajor(smem_u32(sm + C::OFF_KV), kTcKeys, 0);
            const uint64_t dV = D == 128 ? desc_mnmajor128(smem_u32(sm + C::OFF_KV), kTcKeys * 128, 0)
                                         : desc_mnmajor64(smem_u32(sm + C::OFF_KV), 0);
            Ring<NS> ring;
            uint32_t done0 = 0, done1 = 0;             // key tiles of the jobs before, of each tile of rows
            uint32_t held0 = 0, held1 = 0;             // jobs with any
            for (int32_t round = 0;; ++round) {
                wait.for_job(&bar.jfull[round & 1], (round >> 1) & 1);
                if (wait.dead()) break;
                const Job& job = bar.job[round & 1];
                if (!uniform(job.found)) break;
                const Plan& p = job.p;
                const int32_t steps = uniform(p.steps), n0 = uniform(p.n[0]), n1 = uniform(p.n[1]);
                const int32_t keys0 = uniform(p.keys[0] - (p.j0 << kTcKeyShift)),
                              keys1 = uniform(p.keys[1] - (p.j0 << kTcKeyShift));
                const int32_t slots = uniform(p.slot[0] + p.slot[1]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.jempty[round & 1]);
                // The products fill shared memory's bandwidth, and a look at a barrier takes 100 to
                // 200 cycles beside them: the looks at weights are issued among the products before
                // those that need them.  One copy of this code serves both tiles of rows, since the
                // roles compete for the instruction cache.
                bool seen = false;
                uint32_t v = 0;                        // the slot of the step's values
                Ring<NS> vring = ring;                 // that slot and its phase
                if (steps > 0) wait(&bar.full[ring.slot], ring.phase);
                // Steps in the middle, of whole tiles for both tiles of rows: without a question but
                // whether what they need is there.  The few instructions between the products
                // were a fifth of the time (16384 tokens: 3.21 -> 2.77 ms).
                auto steady = [&](int32_t i) {
                    const uint32_t ph0 = (done0 + i) & 1, ph1 = (done1 + i) & 1;
                    auto pv = [&](uint32_t m, uint64_t d) {
#pragma unroll
                        for (uint32_t s = 0; s < kTcKeys / 16; ++s)
                            mma_ts(lead, tmem + C::TM_O + m * D, tmem + C::TM_S + m * kTcKeys + 8 * s,
                                   desc_advance(d, mnmajor_off(s)), id_o, 1);
                    };
                    Ring<NS> kr = ring;                // its keys are behind the step's values
                    kr.next();
                    Ring<NS> vn = kr, kn;              // and the next step's behind them
                    vn.next();
                    kn = vn;
                    kn.next();
                    const uint64_t d = desc_advance(dV, ring.slot * C::SLOT), k = desc_advance(dK, kr.slot * C::SLOT);
                    if (!__all_sync(0xffffffffu, seen)) {
                        wait(&bar.full[ring.slot], ring.phase);
                        wait(&bar.full[kr.slot], kr.phase);
                        wait(&bar.pfull[0], ph0);
                    }
                    fence_after_sync();
                    pv(0, d);
                    commit_if(lead, &bar.ofull[0]);
#pragma unroll
                    for (uint32_t s = 0; s < D / 16; ++s) {
                        if (s == D / 32) seen = mbar_test(&bar.pfull[1], ph1);
                        mma_ss(lead, tmem + C::TM_S, desc_advance(dQ, kmajor_off(kTcRows, s)),
                               desc_advance(k, kmajor_off(kTcKeys, s)), id_s, s > 0);
                    }
                    commit_if(lead, &bar.sfull[0]);
                    wait.after(seen, &bar.pfull[1], ph1);
                    fence_after_sync();
                    pv(1, d);
                    commit_if(lead, &bar.ofull[1]);
                    commit_if(lead, &bar.empty[ring.slot]);
#pragma unroll
                    for (uint32_t s = 0; s < D / 16; ++s) {
                        if (s == D / 32)
                            seen = mbar_test(&bar.pfull[0], ph0 ^ 1) & mbar_test(&bar.full[vn.slot], vn.phase) &
                                   mbar_test(&bar.full[kn.slot], kn.phase);
                        mma_ss(lead, tmem + C::TM_S + kTcKeys, desc_advance(dQ, C::QTILE + kmajor_off(kTcRows, s)),
                               desc_advance(k, kmajor_off(kTcKeys, s)), id_s, s > 0);
                    }
                    commit_if(lead, &bar.sfull[1]);
                    commit_if(lead, &bar.empty[kr.slot]);
                    ring = vn;
                };
                const int32_t middle = min(n0, n1) - 2;
#pragma unroll 1
                for (int32_t i = -1; i < steps; ++i) {
                    if (i >= 1 && i < middle && !wait.dead()) {
                        ring = vring;
                        seen = false;
#pragma unroll 1
                        for (; i < middle && !wait.dead(); ++i) steady(i);
                        // back to the general form: step i's values and the keys behind them
                        wait(&bar.full[ring.slot], ring.phase);
                        v = ring.slot;
                        ring.next();
                        wait(&bar.full[ring.slot], ring.phase);
                        wait.after(seen, &bar.pfull[0], (done0 + i) & 1);
                        seen = true;
                    }
#pragma unroll 1
                    for (int32_t m = 0; m < 2; ++m) {
                        const int32_t n = m ? n1 : n0;
                        const uint32_t s_tm = tmem + C::TM_S + m * kTcKeys, mine = (m ? done1 : done0) + i;
                        if (i >= 0 && i < n) {
                            if (i == 0) wait(&bar.oempty[m], ((m ? held1 : held0) & 1) ^ 1);
                            wait.after(seen, &bar.pfull[m], mine & 1);
                            if (!wait.dead()) {
                                fence_after_sync();
                                const uint64_t d = desc_advance(dV, v * C::SLOT);
                                const int32_t left = (m ? keys1 : keys0) - (i << kTcKeyShift);
                                auto step = [&](uint32_t s) {
                                    mma_ts(lead, tmem + C::TM_O + m * D, s_tm + 8 * s, desc_advance(d, mnmajor_off(s)),
                                           id_o, i > 0 || s > 0);
                                };
                                if (left >= kTcKeys) {
#pragma unroll
                                    for (uint32_t s = 0; s < kTcKeys / 16; ++s) step(s);
                                } else {
#pragma unroll 1
                                    for (uint32_t s = 0; 16 * (int32_t)s < left; ++s) step(s);
                                }
                                commit_if(lead, &bar.ofull[m]);
                            }
                        }
                        if (m && i >= 0 && !wait.dead()) commit_if(lead, &bar.empty[v]);
                        seen = false;
                        if (i + 1 < n) {
                            if (i < 0) wait(&bar.qfull[m], (m ? held1 : held0) & 1);
                            // halfway, a look at the weights of the other tile of rows
                            const int32_t other = m ? i + 1 : i;
                            const bool look = other >= 0 && other < (m ? n0 : n1);
                            if (!wait.dead()) {
                                fence_after_sync();
                                const uint64_t q = desc_advance(dQ, m * C::QTILE), k = desc_advance(dK, ring.slot * C::SLOT);
#pragma unroll
                                for (uint32_t s = 0; s < D / 16; ++s) {
                                    if (s == D / 32 && look) seen = mbar_test(&bar.pfull[m ^ 1], ((m ? done0 : done1) + other) & 1);
                                    mma_ss(lead, s_tm, desc_advance(q, kmajor_off(kTcRows, s)),
                                           desc_advance(k, kmajor_off(kTcKeys, s)), id_s, s > 0);
                                }
                                commit_if(lead, &bar.sfull[m]);
                                if (i + 2 == n) commit_if(lead, &bar.qempty[m]);
                            }
                        }
                    }
                    // the step's keys, then the next one's tiles, while these products run
                    if (i + 1 < steps) {
                        if (!wait.dead()) commit_if(lead, &bar.empty[ring.slot]);
                        ring.next();
                        vring = ring;
                        wait(&bar.full[ring.slot], ring.phase);
                        v = ring.slot;
                        ring.next();
                        if (i + 2 < steps) wait(&bar.full[ring.slot], ring.phase);
                    }
                }
                for (int32_t i = 0; i < slots; ++i) ring.next();
                done0 += n0;
                done1 += n1;
                held0 += n0 > 0;
                held1 += n1 > 0;
            }
            commit_if(lead, &bar.drain);               // no MMA outlives the loop
            mbar_wait(&bar.drain, 0);
            __syncwarp();
        } else {
            // -------------------------------------------------------- outputs from their ring slots
            const int m = warp - C::WARP_STORE;
            uint32_t c = 0, count = 0;
            for (int32_t round = 0;; ++round) {
                wait.for_job(&bar.jfull[round & 1], (round >> 1) & 1);
                if (wait.dead()) break;
                const Job job = bar.job[round & 1];
                if (!job.found) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.jempty[round & 1]);
                const Plan& p = job.p;
                if (p.slot[m]) {
                    const uint32_t at = (c + 2 * p.steps + (m ? p.slot[0] : 0)) % NS;
                    wait.for_job(&bar.staged[m], count++ & 1);
                    if (wait.dead()) break;
                    if (lane == 0) {
                        for (int h = 0; h < HALVES; ++h)
                            tma_store_3d(&maps.out, sm + C::OFF_KV + at * C::SLOT + h * (kTcRows * 128), 64 * h,
                                         job.unit * sh.heads, job.t.row0 + m * sh.tokens);
                        tma_store_wait<true>();
                        mbar_arrive(&bar.empty[at]);
                    }
                    __syncwarp();
                }
                c += 2 * p.steps + p.slot[0] + p.slot[1];
            }
            if (lane == 0) tma_store_wait<false>();
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ softmax
        more_registers<C::REGS_SOFTMAX>();
        const int m = warp >> 2, quad = warp & 3, r = tid & 127;
        const uint32_t lane0 = tmem_addr(tmem, 32 * quad, 0);
        const uint32_t s_tm = lane0 + C::TM_S + m * kTcKeys, o_tm = lane0 + C::TM_O + m * D;
        const int32_t i_tok = r / sh.heads, g = r - i_tok * sh.heads;
        const int32_t token = m * sh.tokens + i_tok;                  // of the job's tokens
        // positive (for a scale of zero as good as zero), so that a masked score stays -infinity
        const float factor = a.scale == 0.f ? 1.2e-38f : fabsf(a.scale) * kAttnLog2e;
        uint32_t c = 0, done = 0;                      // ring slots and key tiles of the jobs before
        for (int32_t round = 0;; ++round) {
            wait.for_job(&bar.jfull[round & 1], (round >> 1) & 1);
            if (wait.dead()) break;
            const Job job = bar.job[round & 1];
            if (!job.found) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.jempty[round & 1]);
            const Plan& p = job.p;
            const AttnTile& t = job.t;
            const int32_t n = m ? p.n[1] : p.n[0];
            const int32_t limit = a.causal ? t.pos0 + token + 1 : t.kv_len;
            const int32_t least = a.causal ? t.pos0 + m * sh.tokens + 1 : t.kv_len;   // any row's
            float ref = -CUDART_INF_F, sum = 0.f;
            for (int32_t i = 0; i < n; ++i) {
                const int32_t key0 = (p.j0 + i) << kTcKeyShift;
                const uint32_t phase = (done + i) & 1;
                wait(&bar.sfull[m], phase);
                fence_after_sync();
                float s[kTcKeys];
#pragma unroll
                for (int k = 0; k < kTcKeys; k += 32) tmem_ld32_start(s_tm + k, s + k);
                tmem_ld_wait(s);
                if (key0 + kTcKeys > least) {
#pragma unroll
                    for (int k = 0; k < kTcKeys; ++k) s[k] = key0 + k < limit ? s[k] : -CUDART_INF_F;
                }
                // The first half's weights from the reference as it is, beside the maximum that may
                // move it: then once more.
                uint32_t w[32];
                float2 add[2];
                auto weigh = [&](int half) {
                    // all scores so far -infinity: nothing to subtract
                    const float base = ref == -CUDART_INF_F ? 0.f : -ref;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const int at = 64 * half + 2 * k;
                        const float2 x = fma2(make_float2(s[at], s[at + 1]), both(factor), both(base));
                        const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                        add[k & 1] = fma2(e, both(1.f), add[k & 1]);
                        w[k] = pack_bf16(e.x, e.y);
                    }
                };
                auto largest = [&] {
                    float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int k = 4; k + 8 <= kTcKeys; k += 8) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) top[x] = max3(top[x], s[k + x], s[k + 4 + x]);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) top[x] = fmaxf(top[x], s[kTcKeys - 4 + x]);
                    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * factor;
                };
                if (i == 0) ref = fmaxf(ref, largest());           // none to begin with (NaN: still none)
                for (;;) {
                    add[0] = add[1] = make_float2(0.f, 0.f);
                    weigh(0);
                    const float most = largest();
                    const bool grown = most > ref + kGrowth;
                    if (!__any_sync(0xffffffffu, grown)) break;
                    const float keep = grown ? exp2f(ref - most) : 1.f;
                    if (grown) ref = most;
                    sum *= keep;
                    if (i > 0) {
                        wait(&bar.ofull[m], phase ^ 1);
                        fence_after_sync();
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            float x[32];
                            tmem_ld32(o_tm + k, x);
#pragma unroll
                            for (int y = 0; y < 32; ++y) x[y] *= keep;
                            tmem_st32(o_tm + k, reinterpret_cast<const uint32_t*>(x));
                        }
                    }
                }
                tmem_st32(s_tm, w);
                weigh(1);
                tmem_st32(s_tm + 32, w);
                sum += add[0].x + add[0].y + add[1].x + add[1].y;
                if (key0 + kTcKeys > p.all) {
                    // value rows past the last key, as far as the product reads (16 at a time)
                    const uint32_t at = c + 2 * i + 1;
                    wait(&bar.full[at % NS], (at / NS) & 1);
                    const int first = p.all - key0, rows = ((first + 15) & ~15) - first;
                    unsigned char* v = sm + C::OFF_KV + at % NS * C::SLOT;
#pragma unroll 1
                    for (int e = r; e < rows * 8 * HALVES; e += 128)
                        *reinterpret_cast<uint4*>(v + (e >> 3) % HALVES * (kTcKeys * 128) +
                                                  (first + (e >> 3) / HALVES) * 128 + (e & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                }
                tmem_st_wait();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.pfull[m]);
            }
            const bool live = i_tok < (m ? p.tokens[1] : p.tokens[0]);
            const int64_t row = (int64_t)(t.row0 + token) * a.Hq + job.unit * sh.heads + g;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            char* ws = static_cast<char*>(a.workspace);
            float* py = a.pieces > 1 ? reinterpret_cast<float*>(ws + attn_pieces_o(a, job.piece)) + row * D : nullptr;
            __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.out) + row * D;
            if (live) {
                const float lse = sum == 0.f ? -CUDART_INF_F : (ref + log2f(sum)) * kAttnLn2;
                if (a.pieces > 1) reinterpret_cast<float*>(ws + attn_pieces_lse(a, job.piece))[row] = lse;
                else if (a.lse != nullptr) a.lse[row] = lse;
            }
            const bool slot = m ? p.slot[1] : p.slot[0];
            if (n > 0) {
                wait(&bar.ofull[m], (done + n - 1) & 1);
                fence_after_sync();
                if (slot) {
                    // through a ring slot: 32 rows of a warp in 16-byte pieces would take a cycle
                    // each of the path that the barriers share
                    const uint32_t at = c + 2 * p.steps + (m ? p.slot[0] : 0);
                    unsigned char* buf = sm + C::OFF_KV + at % NS * C::SLOT;
                    wait(&bar.full[at % NS], (at / NS) & 1);
                    const bool weight = sum != 0.f;        // else zeros, whatever the products gave
#pragma unroll
                    for (int k = 0; k < D; k += 32) {
                        float x[32];
                        tmem_ld32(o_tm + k, x);
#pragma unroll
                        for (int y = 0; y < 32; ++y) x[y] = weight ? x[y] * inv : 0.f;
#pragma unroll
                        for (int y = 0; y < 32; y += 8)
                            *reinterpret_cast<uint4*>(buf + sw128_tile(kTcRows, r, 2 * (k + y))) =
                                make_uint4(pack_bf16(x[y], x[y + 1]), pack_bf16(x[y + 2], x[y + 3]),
                                           pack_bf16(x[y + 4], x[y + 5]), pack_bf16(x[y + 6], x[y + 7]));
                    }
                    fence_async_smem();
                } else {
                    store_row<D>(o_tm, inv, live && sum != 0.f, y, py);
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.oempty[m]);
                    if (slot) mbar_arrive(&bar.staged[m]);
                }
            }
            // no weight: zeros, whatever the products gave
            if (live && sum == 0.f && !slot) {
                if (py != nullptr) {
                    for (int k = 0; k < D; k += 4) *reinterpret_cast<float4*>(py + k) = make_float4(0.f, 0.f, 0.f, 0.f);
                } else {
                    for (int k = 0; k < D; k += 8) *reinterpret_cast<uint4*>(y + k) = make_uint4(0, 0, 0, 0);
                }
            }
            __syncwarp();
            c += 2 * p.steps + p.slot[0] + p.slot[1];
            done += n;
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == C::WARP_MMA) {
        fence_after_sync();
        tmem_dealloc(tmem, C::TM_COLS);
    }
}

template <int D> cudaError_t forward(const AttnArgs& a, cudaStream_t stream)
{
    using C = Cfg<D>;
    const AttnShape sh = attn_shape(kTcRows, a.Hq, a.Hk);
    const int64_t jobs = attn_tiles(a.N, a.T, 2 * sh.tokens) * sh.units * a.splits;
    if (jobs > INT32_MAX) return cudaErrorInvalidValue;
    const int64_t ctas = jobs < sm_count() ? jobs : sm_count();
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    cudaError_t e = encode_heads(&maps.q, a.q, a.T, a.Hq, D, a.q_stride, sh.heads, sh.tokens);
    if (e == cudaSuccess) e = encode_heads(&maps.out, a.out, a.T, a.Hq, D, (int64_t)a.Hq * D, sh.heads, sh.tokens);
    if (a.table == nullptr) {
        if (e == cudaSuccess) e = encode_heads(&maps.k, a.k, a.T, a.Hk, D, a.k_stride, 1, kTcKeys);
        if (e == cudaSuccess) e = encode_heads(&maps.v, a.v, a.T, a.Hk, D, a.v_stride, 1, kTcKeys);
    } else {
        const int page = 1 << a.page_shift, box = page < kTcKeys ? page : kTcKeys;
        const int64_t rows = (int64_t)a.num_pages * a.Hk * page;
        // an empty cache has no page to read: the maps only have to be valid
        const int64_t any = (int64_t)a.T;
        if (e == cudaSuccess) e = encode_rows(&maps.k, rows ? a.k : a.q, true, rows ? rows : any, D, 64, box, true);
        if (e == cudaSuccess) e = encode_rows(&maps.v, rows ? a.v : a.q, true, rows ? rows : any, D, 64, box, true);
    }
    if (e != cudaSuccess) return e;
    auto kern = attn_fwd_tc_kernel<D>;
    static std::atomic<uint64_t> set{0};
    static const cudaError_t registers = check_registers(kern, C::REGS);
    e = registers == cudaSuccess ? allow_smem(kern, C::SMEM, &set) : registers;
    if (e != cudaSuccess) return e;
    return launch_after(kern, launch_config(ctas, C::NT, C::SMEM), stream, a, sh,
                        (int32_t)jobs, maps);
}

}  // namespace

cudaError_t launch_attention_tc(const AttnArgs& a, cudaStream_t stream)
{
    return a.D == 64 ? forward<64>(a, stream) : forward<128>(a, stream);
}

}  // namespace kda
