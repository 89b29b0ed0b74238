// Internal declarations of the attention entry points for several tokens a sequence
// (kda_attention_fwd, kda_attention_bwd, kda_paged_prompt, kda_paged_decode_shared).
//
// Rows.  The query heads of a group (those that share a key-value head) and the tokens
// are packed into one axis: a tile of R tokens and GP heads is R * GP rows, row r being
// token r / GP, head r % GP.  The keys that a tile reads then serve the whole group, and a
// call with one token a sequence still fills its rows.
//
// Order.  A tile's work is its number of key tiles; CTAs are numbered so that the tiles
// with the most come first, whichever sequence they belong to (AttnWalk), and the last
// to start are the shortest.
#pragma once

#include <stdint.h>

#include "kda_paged.cuh"

namespace kda {

struct AttnArgs {
    const void* q;           // [T, Hq, D], tokens q_stride elements apart
    const void* k;           // packed [T, Hk, D] (k_stride), or the cache
    const void* v;
    int32_t q_stride, k_stride, v_stride;
    bool bf16;
    const int32_t* cu;       // [N + 1]
    int32_t N, T, Hq, Hk, D;
    float scale;
    // the paged forms; table == nullptr: keys and values are packed like the queries
    const int32_t* table;    // [N, max_pages]
    const int32_t* kv_lens;  // [N]
    int32_t num_pages, page_shift, max_pages;
    bool causal;             // the last query is the last key's token; else all see all keys
    void* out;               // [T, Hq, D]
    float* lse;              // [T, Hq] or nullptr
    // pieces of the keys' axis, joined by launch_attn_join: [pieces][T, Hq] lse, then
    // [pieces][T, Hq, D] FP32 outputs, behind a header (the number of tokens with a row)
    int32_t splits, pieces;
    void* workspace;
    int32_t* status;
    // backward
    const void* dout;        // [T, Hq, D]
    const float* lse_in;
    float* delta;            // [T, Hq], in the workspace
    void* dq;
    void* dk;
    void* dv;
    // test hook (kda_test_set_fault): the kernel that it names withholds an arrival in CTA 0
    int32_t fault;
};

// Bytes before the pieces' statistics.
constexpr int64_t kAttnHeader = 256;
__host__ __device__ inline int64_t attn_pieces_lse(const AttnArgs& a, int32_t piece)
{
    return kAttnHeader + (int64_t)piece * a.T * a.Hq * 4;
}
__host__ __device__ inline int64_t attn_pieces_o(const AttnArgs& a, int32_t piece)
{
    const int64_t rows = (int64_t)a.T * a.Hq;
    return kAttnHeader + ((int64_t)a.pieces * rows * 4 + 255) / 256 * 256 + piece * rows * a.D * 4;
}

// How a call's rows are cut into tiles.
struct AttnShape {
    int32_t tokens;          // of a CTA's tile
    int32_t heads;           // query heads of a tile
    int32_t parts;           // tiles of heads per group
    int32_t units;           // Hk * parts
};

cudaError_t launch_attention_tc(const AttnArgs& a, cudaStream_t stream);      // BF16
cudaError_t launch_attention_bwd_tc(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attention(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attention_bwd(const AttnArgs& a, cudaStream_t stream);
int64_t attention_bwd_workspace_bytes(int32_t N, int32_t T, int32_t Hq, int32_t Hk, int32_t D);
cudaError_t launch_attn_join(const AttnArgs& a, cudaStream_t stream);
// Pieces of the keys' axis for a call whose sequences have at most kv_most keys.
int32_t attn_splits(bool bf16, int32_t N, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t kv_most);

// ---------------------------------------------------------------- device
struct AttnTile {
    int32_t n;               // sequence
    int32_t index;           // of the tile in it
    int32_t row0, tokens;    // first packed token, and how many
    int32_t seq0, seq_tokens;    // the sequence's first packed token, and its tokens
    int32_t kv_len;          // keys of the sequence
    int32_t pos0;            // position of the tile's first token (below 0: it sees no key)
};

// The sequence's keys; a length that the table or the cache cannot hold counts as none.
__device__ __forceinline__ int32_t attn_kv_len(const AttnArgs& a, int32_t n, int32_t tokens)
{
    if (a.table == nullptr) return tokens;
    const int32_t L = a.kv_lens[n];
    const int64_t most = (int64_t)a.max_pages << a.page_shift;
    if (L < 0 || L > most || (L > 0 && a.num_pages == 0)) {
        report_status(a.status, KDA_ERR_DEVICE_ARG);
        return 0;
    }
    return L;
}

// Of a sequence of m tokens and L keys, cut into nt tiles of `tokens`: the first tile that
// has more than d key tiles of 2^key_shift (nt: none has).
__device__ __forceinline__ int32_t attn_deeper(int32_t m, int32_t L, int32_t nt, bool causal, int32_t tokens,
                                               int key_shift, int32_t d)
{
    if (d < 0) return 0;
    const int64_t lim = (int64_t)d << key_shift;
    if (L <= lim) return nt;
    if (!causal) return 0;
    const int64_t x = lim - ((int64_t)L - m);          // tokens whose keys end within lim
    return x <= 0 ? 0 : min(nt, (int32_t)((uint32_t)x / (uint32_t)tokens));
}

// The tiles of a call in the order of falling work, walked by one whole warp: next(item) for
// rising items.  Tiles that have the same number of key tiles are a level; a walk keeps its
// place in one, so that a call with thousands of short sequences looks at each once.  The
// first 32 sequences stay in the lanes' registers: a look at memory takes several hundred
// cycles beside the products.
struct AttnWalk {
    int32_t tokens, key_shift;
    bool bad;                // bad offsets (reported): there are no tiles
    int32_t level;           // tiles of `level` key tiles
    int32_t first, behind;   // the level's first item, and the next one's
    int32_t base, passed;    // sequences from `base` on; items of the level before them
    struct Sequence {
        int32_t c0, m, L, nt;        // first packed token, tokens, keys, tiles
    } mine;                  // of sequence `lane`

    __device__ __forceinline__ Sequence look(const AttnArgs& a, int32_t n) const
    {
        Sequence s;
        s.c0 = a.cu[n];
        s.m = (int32_t)((uint32_t)a.cu[n + 1] - (uint32_t)s.c0);
        s.L = attn_kv_len(a, n, s.m);
        s.nt = (int32_t)(((uint32_t)s.m + tokens - 1) / (uint32_t)tokens);
        return s;
    }
    // the sequence base + lane; none: without tiles
    __device__ __forceinline__ Sequence at(const AttnArgs& a, int32_t base_) const
    {
        const int32_t n = base_ + (threadIdx.x & 31);
        return base_ == 0 ? mine : n < a.N ? look(a, n) : Sequence{0, 0, 0, 0};
    }
    // its tiles that have more than d key tiles
    __device__ __forceinline__ int32_t count(const AttnArgs& a, const Sequence& s, int32_t d) const
    {
        return s.nt - attn_deeper(s.m, s.L, s.nt, a.causal, tokens, key_shift, d);
    }
    __device__ __forceinline__ int32_t total(const AttnArgs& a, int32_t d) const
    {
        int32_t x = count(a, mine, d);
        for (int32_t b = 32; b < a.N; b += 32) x += count(a, at(a, b), d);
        return (int32_t)__reduce_add_sync(0xffffffffu, (unsigned)x);
    }
    __device__ __forceinline__ AttnWalk(const AttnArgs& a, int32_t tile_tokens, int shift)
        : tokens(tile_tokens), key_shift(shift), bad(false), level(0), first(0), behind(0), base(0), passed(0),
          mine{0, 0, 0, 0}
    {
        const int lane = threadIdx.x & 31;
        int32_t deepest = 0;
        for (int32_t n = lane; n < a.N; n += 32) {
            const int32_t c1 = a.cu[n + 1];
            const Sequence s = look(a, n);
            // the offsets themselves: a difference of bad ones may wrap to a length
            bad |= s.c0 < 0 || c1 < s.c0 || c1 > a.T || (n == 0 && s.c0 != 0);
            deepest = max(deepest, s.L);
            if (n == lane) mine = s;
        }
        bad = __any_sync(0xffffffffu, bad);
        if (bad && lane == 0) report_status(a.status, KDA_ERR_DEVICE_ARG);
        deepest = __reduce_max_sync(0xffffffffu, deepest);
        level = (int32_t)(((int64_t)deepest + (1 << key_shift) - 1) >> key_shift) + 1;   // above the first
    }
    __device__ __forceinline__ static void set(AttnTile& t, const Sequence& s, int32_t index, int32_t tokens)
    {
        t.index = index;
        t.seq0 = s.c0;
        t.seq_tokens = s.m;
        t.row0 = s.c0 + index * tokens;
        t.tokens = min(tokens, s.m - index * tokens);
        t.kv_len = s.L;
        t.pos0 = s.L - s.m + index * tokens;
    }
    // false: there is no such tile
    __device__ __forceinline__ bool next(const AttnArgs& a, int32_t item, AttnTile& t)
    {
        if (bad) return false;
        if (a.N == 1) {
            // one sequence: the tiles from its end (a search costs a short call a microsecond)
            const Sequence s = {__shfl_sync(0xffffffffu, mine.c0, 0), __shfl_sync(0xffffffffu, mine.m, 0),
                                __shfl_sync(0xffffffffu, mine.L, 0), __shfl_sync(0xffffffffu, mine.nt, 0)};
            if (item >= s.nt) return false;
            t.n = 0;
            set(t, s, s.nt - 1 - item, tokens);
            return true;
        }
        if (item >= behind) {
            // The item has the least d with at most `item` tiles of more than d key tiles; level - 1
            // is one.  Down from there in growing steps, then by halves.
            int32_t hi = level - 1, hi_total = behind, lo = hi - 1, step = 1;
            if (hi < 0) return false;
            int32_t lo_total = total(a, lo);
            while (lo_total <= item) {
                if (lo < 0) return false;
                hi = lo;
                hi_total = lo_total;
                step *= 2;
                lo = max(hi - step, -1);
                lo_total = total(a, lo);
            }
            while (hi - lo > 1) {
                const int32_t mid = (lo + hi) >> 1, x = total(a, mid);
                if (x <= item) {
                    hi = mid;
                    hi_total = x;
                } else {
                    lo = mid;
                    lo_total = x;
                }
            }
            level = hi;
            first = hi_total;
            behind = lo_total;
            base = passed = 0;
        }
        int32_t rank = item - first - passed;
        const int lane = threadIdx.x & 31;
        for (;; base += 32) {
            if (base >= a.N) return false;             // lengths that changed meanwhile
            const Sequence s = at(a, base);
            const int32_t tiles = count(a, s, level - 1) - count(a, s, level);
            int32_t upto = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const unsigned past = __ballot_sync(0xffffffffu, upto > rank);
            if (past) {
                const int who = __ffs(past) - 1;
                auto of = [&](int32_t x) { return __shfl_sync(0xffffffffu, x, who); };
                rank -= of(upto - tiles);
                const int32_t begin = of(s.nt - count(a, s, level - 1)), m = of(s.m);
                t.n = base + who;
                set(t, Sequence{of(s.c0), m, of(s.L), 0}, begin + rank, tokens);
                return true;
            }
            const int32_t all = __shfl_sync(0xffffffffu, upto, 31);
            rank -= all;
            passed += all;
        }
    }
};

// Kernels that start a CTA a tile take the tiles of more sequences than this without the order,
// since every CTA would look at all of them several times.  32768 tokens in equal sequences, FP32 forward
// (4 heads of 64 channels) and BF16 backward (16 heads of 128): 256 sequences 159 -> 129 and 362 -> 335 us,
// 1024 sequences 212 -> 96 and 752 -> 430, 4096 sequences 2.1 -> 0.28 and 6.4 -> 1.7 ms.  With one sequence of a
// quarter of the tokens behind 127 short ones the order is worth 3% (FP32 1084 us, 1119 without).
constexpr int32_t kAttnOrdered = 128;

// Whether the offsets of a call with more are bad, by all threads of a CTA.
__device__ __forceinline__ bool attn_bad(const AttnArgs& a)
{
    int bad = 0;
    for (int32_t n = threadIdx.x; n < a.N; n += blockDim.x) {
        const int32_t c0 = a.cu[n], c1 = a.cu[n + 1];
        bad |= c0 < 0 || c1 < c0 || c1 > a.T || (n == 0 && c0 != 0);
        if (a.table != nullptr) attn_kv_len(a, n, 0);
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) report_status(a.status, KDA_ERR_DEVICE_ARG);
    return bad != 0;
}
// Its tile `item`, by a whole warp: sequence n has the items from cu[n] / tokens + n on, one or two
// of which may be no tiles.
__device__ __forceinline__ bool attn_place(const AttnArgs& a, int32_t item, int32_t tokens, AttnTile& t)
{
    const int lane = threadIdx.x & 31;
    auto from = [&](int32_t n) { return a.cu[n] / tokens + n; };
    int32_t lo = 0, hi = a.N;                  // from(lo) <= item, and so for none from hi on
    while (hi - lo > 1) {
        const int32_t step = (hi - lo + 31) / 32, n = lo + step * lane;
        const int32_t k = 31 - __clz(__ballot_sync(0xffffffffu, n == lo || (n < hi && from(n) <= item)));
        lo += step * k;
        hi = min(hi, lo + step);
    }
    AttnWalk::Sequence s;
    s.c0 = a.cu[lo];
    s.m = a.cu[lo + 1] - s.c0;
    s.L = attn_kv_len(a, lo, s.m);
    s.nt = (s.m + tokens - 1) / tokens;
    const int32_t index = s.nt - 1 - (item - from(lo));
    t.n = lo;
    if (index >= 0) AttnWalk::set(t, s, index, tokens);
    return index >= 0;
}
// Tile `item` alone; `bad`: of attn_bad.
__device__ __forceinline__ bool attn_find(const AttnArgs& a, bool bad, int32_t item, int32_t tokens, int key_shift,
                                          AttnTile& t)
{
    if (a.N > kAttnOrdered) return !bad && attn_place(a, item, tokens, t);
    AttnWalk w(a, tokens, key_shift);
    return w.next(a, item, t);
}

// Keys that the tile's last token sees.
__device__ __forceinline__ int32_t attn_keys(const AttnArgs& a, const AttnTile& t)
{
    return a.causal ? max(0, t.pos0 + t.tokens) : t.kv_len;
}

// The cache row (of num_pages * Hk * page_size) of head hk's token `at` of sequence n.  An
// entry outside the cache is reported and read as page 0.
__device__ __forceinline__ int64_t attn_page_row(const AttnArgs& a, int32_t n, int32_t hk, int32_t at)
{
    int32_t page = a.table[(int64_t)n * a.max_pages + (at >> a.page_shift)];
    if ((uint32_t)page >= (uint32_t)a.num_pages) {
        report_status(a.status, KDA_ERR_DEVICE_ARG);
        page = 0;
    }
    return (((int64_t)page * a.Hk + hk) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
}

}  // namespace kda
