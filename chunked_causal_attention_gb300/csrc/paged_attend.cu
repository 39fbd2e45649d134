// Attention of the newest tokens, one or a chunk of many a sequence, over the paged
// cache, on the 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
//   s_rj = scale q_r . k_j,   O_r = sum_{j seen by r} 2^(s2_rj - m_r) v_j / l_r,   s2 = s log2 e
//
// Bounds. A decode step reads every key and value once, 4 n Hkv D bytes, and is bound by
// memory. A chunk of many tokens does 4 D operations a (row, slot) pair, but its pace is
// that of the one softmax warpgroup's loop (scores out of TMEM, weights back into it, the
// hand-over to the next product): 2048 tokens over 32K slots take an SM 0.74 us a key tile
// at 64 dims, where the products are 0.28 us, and 0.84 at 128 dims, where they are 0.57;
// the tensor pipe is busy 36% and 67% of the time. Repeated for seconds, 128 dims reach the board's
// power limit as well (704 -> 754 us at a median of 1800 MHz); 64 dims do not (619 -> 621,
// 2070 MHz).
//
// Rows. The G = H / Hkv query heads that share a key/value head read the same slots, so
// a tile of 128 rows is 128 / G tokens of all G heads (of up to 128 of them): a decode
// step's rows are one tile a sequence and key/value head, and a chunk reads its keys
// once for G heads. One TMA box brings the tile's queries, tokens by heads by 64 dims.
// The products are done for all 128 rows whatever their number: 0.56 us a tile of 128
// slots and 128 dims, whose 64 KB take an SM 1.4 us to get from memory when all do.
//
// Work. A unit is one row tile of one key/value head; it reads the slots up to its last
// token. The lengths are on the device, so a warp of every block derives the same list
// of items from them: units of more than C key tiles are cut into equal parts, C by
// weighing a few shares of an SM's work against each other (make_list). The parts'
// (O, LSE) go to the workspace and merge_kernel joins them in order, so the result does
// not depend on timing. Items of one key/value head and part follow each other in the
// list, so blocks that run together read the same keys from L2; a block takes its first
// item by its number and the others from a queue.
//
// Roles of a block's warps: 0 takes items, looks up pages (32 boxes' entries of the table
// at a time, a lane each, one window ahead) and issues the TMA loads, a box for each page
// (or part of one) and 64 dims; 1 issues the MMAs; 2 and 3 clear what no row may see in
// a tile of V (below); 4 to 7 do the softmax, a row a thread, as in the forward.
//
// Small pages. A TMA copy takes about 45 ns of the unit's time however small its box is:
// pages of 16 slots make 32 boxes a key tile, 1.5 us. There (GATHER) warps 2 and 3 bring
// V by 16-byte copies, one half of a tile each, and TMA brings K alone. 2048 tokens over
// 32K slots, by TMA and with the copies: 128 dims, pages of 16 1337 and 857 us, of 32 888
// and 770, of 64 707 and 772; 64 dims 888 and 673, 659 and 669, 618 and 669; 256 dims, 4
// heads: 1339 and 858, 1021 and 745, 913 and 739 (where pages of 64, which have 32 boxes of
// K and V a tile as well, would be better off with the copies).
//
// Masked slots. A masked score is replaced before the maximum, so K may hold anything
// there. But weight 0 times a NaN or an infinity in V would reach the sum, so in tiles
// that some row does not see whole, warps 2 and 3 zero the rows of V behind the last
// slot, and replace values that are not finite in rows that only some tokens see; these
// are added to the rows that do see them at the end. Pages behind the last one are
// loaded from beyond the tensor map's edge: zeros.
//
// Measured: one token over 1M slots of 8 heads 587 us (7.3 TB/s), of 48 sequences of 13K
// slots on average over pages of 16 390 us (6.7 TB/s), of 512 sequences of 1300 slots 470 us
// (5.9 TB/s), over 1000 slots 12.5 us; 2048 tokens over 32K slots, 32 heads in groups of 4,
// 684 to 725 us (1470 to 1560 TFLOP/s).
#include <algorithm>

#include "kv4_device.cuh"
#include "paged.h"
#include "tc_common.cuh"

namespace attn {
namespace {

using namespace tc;
using kv4::grid_go;
using kv4::grid_wait;
using kv4::launch_early;

constexpr int kThreads = 256;
constexpr int kItemsPerSm = 8;                 // the smallest items are an eighth of an SM's work
// What an item takes beside its key tiles, in those: 2 to 5 us of filling and draining the pipeline.
constexpr float kItemTiles = 3.f;
// What a row of a partial takes to write and read again, in key tiles. Chunks of four prompts 203 us and 2048
// tokens over 32K slots 752; with half of it 213 and 752, with three times 202 and 775.
constexpr float kRowTiles = 1.f / 16;
constexpr int kGatherPage = 32;                // pages up to which V is copied (see above)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;
constexpr uint32_t kColO = 256;
constexpr float kLag = 8.f;                    // how far (log2) a tile's maximum may pass the running one
// Rows of a warp up to which it may not: the largest weight is then 1, which bf16 holds exactly, so that a row that one
// slot dominates is not off by that weight's rounding: single tokens are off by 1.8e-3 relative to 64 bits instead of
// 2.2e-3 to 2.4e-3 (the output's rounding alone: 1.7e-3), for 1% of the batch's time and 4% of the mixed one's. For many
// rows O would be rescaled at most tiles.
constexpr int kExactRows = 16;

// What the launch derives from the shapes.
struct Tiling {
    int32_t heads, blocks;     // query heads of a row tile, and how many such tiles a key/value head's heads make
    int32_t group;             // query heads of a key/value head
    int32_t units;             // units of a row tile's tokens: key/value heads by blocks of heads
    int32_t tok, few;          // tokens of a row tile, and of the small box that brings fewer
    FastDiv by_tok;
    int32_t wide;              // rows of O may be stored 32 bytes at a time
    int32_t head_major;        // rows of a tile: head * tokens of the box + token, or token * heads + head
    int32_t box;               // slots of a TMA box of K and V
    int32_t part_rows;         // rows of a partial
    int64_t part_floats;       // floats of a partial: rows of D, then their LSEs (base 2)
    int32_t sms;
};

__host__ __device__ constexpr int block_n(int d) { return d > 128 ? 64 : 128; }     // slots of a key tile
__host__ __device__ constexpr int stages(int d) { return d > 128 ? 2 : d > 64 ? 3 : 6; }

Tiling tiling(const PagedGeom& c, const Geom& g) {
    Tiling t;
    const int32_t G = g.H / c.Hkv;
    t.heads = std::min(G, kTile);
    t.blocks = (G - 1) / t.heads + 1;
    t.group = G;
    t.units = c.Hkv * t.blocks;
    t.tok = kTile / t.heads;
    t.by_tok = FastDiv::of((uint32_t)t.tok);
    t.few = std::max(1, std::min(t.tok, 16 / t.heads));
    t.wide = t.head_major = 0;
    t.box = std::min(c.page(), block_n(g.D));
    t.part_rows = (int32_t)std::min<int64_t>(t.tok, g.T) * t.heads;
    t.part_floats = ((int64_t)t.part_rows * (g.D + 1) + 31) / 32 * 32;
    t.sms = device_sm_count();
    return t;
}

// ------------------------------------------------------------------ the work list

struct Seq {
    int32_t q0, nq, n;         // first packed token, tokens, slots in use
};

// Offsets that leave [0, T] or descend, each as the nearest one in [the one before it, T]: sequences have no token in
// common then. By one warp of every block, all of which write the same to the workspace.
__device__ __noinline__ const int32_t* offsets_in_order(const PagedAttendArgs& a) {
    const int lane = threadIdx.x & 31;
    int32_t from = 0;
    for (int32_t base = 0; base <= a.B; base += 32) {
        int32_t x = base + lane <= a.B ? max(from, min(a.cu[base + lane], a.g.T)) : from;
        for (int m = 1; m < 32; m <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, x, m);
            if (lane >= m) x = max(x, y);
        }
        if (base + lane <= a.B) a.offsets[base + lane] = x;
        from = __shfl_sync(0xffffffffu, x, 31);
    }
    __syncwarp();
    return a.offsets;
}

// Sequence b by the offsets cu; sets `bad` where they are not in order.
__device__ __forceinline__ Seq seq_of(const PagedAttendArgs& a, const int32_t* cu, int32_t b, bool& bad) {
    Seq s;
    int32_t hi;
    if (cu) {
        s.q0 = cu[b];
        hi = cu[b + 1];
        if (!(0 <= s.q0 && s.q0 <= hi && hi <= a.g.T)) {
            set_error(a.status, ATTN_E_BOUNDS);
            bad = true;
            s.q0 = max(0, min(s.q0, a.g.T));
            hi = max(s.q0, min(hi, a.g.T));
        }
    } else {
        s.q0 = b * a.each;
        hi = s.q0 + a.each;
    }
    s.nq = hi - s.q0;
    const int32_t most = a.max_pages << a.c.shift;
    s.n = a.lens[b];
    if (s.n < 0 || s.n > most) {
        set_error(a.status, ATTN_E_BOUNDS);
        s.n = max(0, min(s.n, most));
    }
    return s;
}

__device__ __forceinline__ int32_t row_tiles_of(const Tiling& t, int32_t nq) {
    return nq > 0 ? (int32_t)t.by_tok.div((uint32_t)(nq - 1)) + 1 : 0;
}

// Units of a sequence, and the key tiles of its longest.
__device__ __forceinline__ int32_t units_of(const Tiling& t, const Seq& s) { return t.units * row_tiles_of(t, s.nq); }
template <int BN>
__device__ __forceinline__ int32_t tiles_of(const Seq& s) { return max(1, (s.n + BN - 1) / BN); }

// n / d for whole numbers, where d is often one.
__device__ __forceinline__ int32_t quotient(int32_t n, int32_t d) { return d == 1 ? n : (int32_t)((uint32_t)n / (uint32_t)d); }

__device__ __forceinline__ int32_t parts_of(int32_t tiles, int32_t C) { return tiles > C ? (tiles - 1) / C + 1 : 1; }

// The list as the lanes of a warp hold it: each a run of `per` sequences.
struct List {
    int32_t first, items;      // the run's first item, and how many it has
    int32_t parts;             // partials of the runs before
    Seq seq;                   // the run's sequence, where it is one
    const int32_t* cu;         // offsets in order: the caller's, or what was made of them
    int32_t per;
    int32_t C;                 // most key tiles of an item
    int32_t whole, tail;       // one sequence's rounds: units left whole, parts of the others; tail 0: all are cut by C
    int32_t n_items;
};

// Where in a run of several sequences the last item was found: 32 sequences from b on, items and partials of those
// before. A block's items come in the order of the list, so it goes through every run once: one token of each of 65536
// sequences of up to 60 slots and 8 heads 20.0 ms, and 56.8 by looking from the run's start every time.
struct Found {
    int32_t run, b, items, parts;
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// Sizes of an item that are weighed against each other, in shares of an SM's work. With one alone, of the whole work: five
// tokens of 8 sequences 17.8 us against 17.1 and single tokens of 20 sequences 198 against 187.5, but of 48 381 against 390
// and the mixed batch 110 against 114; of an eighth: 28.1, 189, 390, 139, chunks of four prompts 225 against 193. With four
// (1/8, 1/3, 1, 2): 17.6 and 189, the others within 1%.
constexpr int kTry = 8;
__constant__ const float kShares[kTry] = {1.f / kItemsPerSm, 0.2f, 1.f / 3, 0.5f, 1.f, 1.25f, 1.5f, 2.f};

// How to cut W key tiles of work, by a warp: sets C, whole and tail.
template <int BN>
__device__ __forceinline__ void weigh(const PagedAttendArgs& a, const Tiling& t, float W, List& L) {
    const int lane = threadIdx.x & 31;
    // Of several sizes the one that is done first, in key tiles: by full rounds of the longest item, or as a queue
    // hands items out, whichever is less. A lane takes one size and a quarter of the sequences.
    const float sms = (float)t.sms;
    const float size = fmaxf(1.f, ceilf(__fdividef(W, sms) * kShares[lane & (kTry - 1)]));
    float n_items = 0.f, extra = 0.f, most = 0.f;
    bool bad;
    for (int32_t base = 0; base < a.B; base += 32) {
        const Seq s = L.per == 1 ? L.seq : base + lane < a.B ? seq_of(a, L.cu, base + lane, bad) : Seq{0, 0, 0};
        const float units = (float)units_of(t, s), tiles = (float)tiles_of<BN>(s);
        const float rows = (float)(min(s.nq, t.tok) * t.heads) * kRowTiles;
#pragma unroll 1
        for (int i = 0; i < min(32, a.B - base); i += 32 / kTry) {
            const float u = __shfl_sync(0xffffffffu, units, i + lane / kTry), n = __shfl_sync(0xffffffffu, tiles, i + lane / kTry);
            const float p = ceilf(__fdividef(n, size));
            n_items += u * p;
            const float each = __shfl_sync(0xffffffffu, rows, i + lane / kTry);
            if (p > 1.f) extra += u * p * each;
            if (u > 0.f) most = fmaxf(most, ceilf(__fdividef(n, p)));
        }
    }
#pragma unroll
    for (int m = kTry; m < 32; m <<= 1) {
        n_items += __shfl_xor_sync(0xffffffffu, n_items, m);
        extra += __shfl_xor_sync(0xffffffffu, extra, m);
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
    }
    const float rounds = ceilf(__fdividef(n_items, sms)) * (most + kItemTiles);
    const float queue = __fdividef(W + n_items * kItemTiles, sms) + most;
    float time = fminf(rounds, queue) + __fdividef(extra, sms), C = size;
#pragma unroll
    for (int m = 1; m < kTry; m <<= 1) {
        const float time2 = __shfl_xor_sync(0xffffffffu, time, m), C2 = __shfl_xor_sync(0xffffffffu, C, m);
        if (time2 < time || (time2 == time && C2 < C)) {
            time = time2;
            C = C2;
        }
    }
    L.C = (int32_t)fminf(C, 1073741824.f);
    // One sequence's units are about equal: as many as make full rounds may stay whole, and those of the last round
    // be cut into a few parts (a lane each number), which leaves fewer partials to write and join.
    const int32_t alone = units_of(t, L.seq);
    const uint32_t have = __ballot_sync(0xffffffffu, alone > 0);
    const int32_t at = max(0, __ffs(have) - 1), units = __shfl_sync(0xffffffffu, alone, at), left = units % t.sms;
    if (L.per == 1 && __popc(have) == 1 && units > t.sms && left > 0) {
        const int32_t tiles = __shfl_sync(0xffffffffu, tiles_of<BN>(L.seq), at);
        const float n = (float)tiles, p = (float)min((lane & (kTry - 1)) + 1, tiles), cut = (float)left * p;
        float rounds2 = (float)(units / t.sms) * (n + kItemTiles) +
                        ceilf(__fdividef(cut, sms)) * (ceilf(__fdividef(n, p)) + kItemTiles);
        if (p > 1.f) rounds2 += __fdividef(cut * (float)kTile * kRowTiles, sms);
        int32_t best = (int32_t)p;
#pragma unroll
        for (int m = 1; m < kTry; m <<= 1) {
            const float other = __shfl_xor_sync(0xffffffffu, rounds2, m);
            const int32_t best2 = __shfl_xor_sync(0xffffffffu, best, m);
            if (other < rounds2 || (other == rounds2 && best2 < best)) {
                rounds2 = other;
                best = best2;
            }
        }
        if (rounds2 < time) {
            L.whole = units - left;
            L.tail = best;
        }
    }
}

// By one warp. `tell`: write a.cuts for the merge kernel.
template <int BN>
__device__ __forceinline__ List make_list(const PagedAttendArgs& a, const Tiling& t, bool tell) {
    const int lane = threadIdx.x & 31;
    List L;
    L.per = (a.B + 31) / 32;
    const int32_t b0 = (int32_t)min((int64_t)lane * L.per, (int64_t)a.B);
    const int32_t b1 = (int32_t)min((int64_t)b0 + L.per, (int64_t)a.B);
    float W;
    L.cu = a.cu;
    while (true) {
        bool bad = false;
        W = 0.f;
        L.seq = Seq{0, 0, 0};
#pragma unroll 4
        for (int32_t b = b0; b < b1; ++b) {
            L.seq = seq_of(a, L.cu, b, bad);
            W += (float)units_of(t, L.seq) * (float)tiles_of<BN>(L.seq);
        }
        if (L.cu != a.cu || !__any_sync(0xffffffffu, bad)) break;
        L.cu = offsets_in_order(a);                      // and once more
    }
    W = warp_sum(W);
    L.C = 1;
    L.whole = L.tail = 0;
    if (W > (float)t.sms) weigh<BN>(a, t, W, L);          // less work is cut into single tiles
    int32_t items = 0, parts = 0, longest = 0;
    bool bad;
    for (int32_t b = b0; b < b1; ++b) {
        if (L.per > 1) L.seq = seq_of(a, L.cu, b, bad);
        const int32_t tiles = tiles_of<BN>(L.seq), p = parts_of(tiles, L.C), n = units_of(t, L.seq);
        items += n * p;
        if (p > 1) parts += n * p;
        longest = max(longest, (tiles - 1) / p + 1);
    }
    if (L.tail && items) {
        items = L.whole + (units_of(t, L.seq) - L.whole) * L.tail;
        parts = L.tail > 1 ? items - L.whole : 0;
    }
    int32_t parts_to = parts;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, parts_to, m);
        if (lane >= m) parts_to += y;
    }
    // the runs with the longest items go first, so that the last ones to end are short
    L.first = 0;
    int32_t items_all = 0;
    for (int i = 0; i < min(32, a.B); ++i) {
        const int32_t other = __shfl_sync(0xffffffffu, longest, i), n = __shfl_sync(0xffffffffu, items, i);
        if (other > longest || (other == longest && i < lane)) L.first += n;
        items_all += n;
    }
    const int32_t parts_all = __shfl_sync(0xffffffffu, parts_to, 31);
    // a list of more parts than the workspace holds is not worked off
    const bool fits = parts_all <= a.max_parts;
    if (!fits) set_error(a.status, ATTN_E_BOUNDS);
    L.n_items = fits ? items_all : 0;
    L.items = items;
    L.parts = fits ? parts_to - parts : 0;
    if (tell) {
        int32_t before = parts_to - parts;
        for (int32_t b = b0; b < b1; ++b) {
            if (L.per > 1) L.seq = seq_of(a, L.cu, b, bad);
            const int32_t p = !fits ? 1 : L.tail ? L.tail : parts_of(tiles_of<BN>(L.seq), L.C);
            a.cuts[b] = make_int4(p > 1 ? before : 0, p, L.whole, L.cu != a.cu);
            if (p > 1) before += units_of(t, L.seq) * p;
        }
    }
    return L;
}

// An item as its consumers read it from shared memory.
struct Item {
    int32_t tiles;             // key tiles; -1: no more work
    int32_t k0;                // first slot
    int32_t tok0, toks;        // first packed token, tokens
    int32_t head0, heads;      // first query head, heads
    int32_t seen;              // slots that the first token sees
    int32_t n;                 // slots in use
    int32_t part;              // partial that it writes, -1: the output
    int32_t box;               // tokens of the box that brought its queries
    int32_t b, hk;
};
static_assert(sizeof(Item) == 48, "Item layout");

// Item w of the list, by a whole warp; false if the lengths changed since the list was made.
template <int BN>
__device__ __forceinline__ bool find_item(const PagedAttendArgs& a, const Tiling& t, const List& L, Found& at, int32_t w,
                                          Item& it) {
    const int lane = threadIdx.x & 31;
    const uint32_t here = __ballot_sync(0xffffffffu, w >= L.first && w - L.first < L.items);
    if (!here) return false;
    const int32_t run = __ffs(here) - 1;
    int32_t x = w - __shfl_sync(0xffffffffu, L.first, run), part0 = __shfl_sync(0xffffffffu, L.parts, run);
    int32_t b = run * L.per;
    Seq s{__shfl_sync(0xffffffffu, L.seq.q0, run), __shfl_sync(0xffffffffu, L.seq.nq, run), __shfl_sync(0xffffffffu, L.seq.n, run)};
    if (L.per > 1) {
        const int32_t end = (int32_t)min((int64_t)b + L.per, (int64_t)a.B);
        bool found = false;
        if (at.run != run || x < at.items) at = Found{run, b, 0, 0};
        b = at.b;
        x -= at.items;
        part0 += at.parts;
        for (; b < end; b += 32) {
            int32_t items = 0, cut = 0;
            s = Seq{0, 0, 0};
            if (b + lane < end) {
                bool bad;
                s = seq_of(a, L.cu, b + lane, bad);
                const int32_t p = parts_of(tiles_of<BN>(s), L.C);
                items = units_of(t, s) * p;
                cut = p > 1 ? items : 0;
            }
            int32_t items_to = items, cut_to = cut;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int32_t u = __shfl_up_sync(0xffffffffu, items_to, m), v = __shfl_up_sync(0xffffffffu, cut_to, m);
                if (lane >= m) {
                    items_to += u;
                    cut_to += v;
                }
            }
            const uint32_t past = __ballot_sync(0xffffffffu, items_to > x);
            if (past) {
                const int f = __ffs(past) - 1;
                x -= __shfl_sync(0xffffffffu, items_to - items, f);
                part0 += __shfl_sync(0xffffffffu, cut_to - cut, f);
                s = Seq{__shfl_sync(0xffffffffu, s.q0, f), __shfl_sync(0xffffffffu, s.nq, f), __shfl_sync(0xffffffffu, s.n, f)};
                b += f;
                found = true;
                break;
            }
            const int32_t all = __shfl_sync(0xffffffffu, items_to, 31), all_cut = __shfl_sync(0xffffffffu, cut_to, 31);
            x -= all;
            part0 += all_cut;
            at = Found{run, b + 32, at.items + all, at.parts + all_cut};
        }
        if (!found) return false;
    }
    if (b >= a.B) return false;
    const int32_t row_tiles = row_tiles_of(t, s.nq), units = units_of(t, s);
    if (x < 0 || units == 0) return false;
    int32_t parts, p, u, r;                              // u: key/value head and block of heads; r: row tile, the last first
    if (L.tail) {
        const bool whole = x < L.whole;
        const int32_t y = x - L.whole, left = units - L.whole;
        if (left <= 0) return false;
        p = whole ? 0 : y / left;
        const int32_t unit = whole ? x : L.whole + y - p * left;
        parts = whole ? 1 : L.tail;
        u = unit / row_tiles;
        r = unit - u * row_tiles;
        if (!whole) x = y;
    } else {
        // head, part, row tile: blocks that run together read the same part
        parts = parts_of(tiles_of<BN>(s), L.C);
        const int32_t y = quotient(x, row_tiles);
        r = x - y * row_tiles;
        u = quotient(y, parts);
        p = y - u * parts;
    }
    if (u >= t.units || p >= parts || (parts > 1 && part0 + x >= a.max_parts)) return false;
    const int32_t rt = row_tiles - 1 - r, hk = quotient(u, t.blocks), hb = u - hk * t.blocks;
    const int32_t G = t.group, i0 = rt * t.tok;
    it.tok0 = s.q0 + i0;
    it.toks = min(t.tok, s.nq - i0);
    it.head0 = hk * G + hb * t.heads;
    it.heads = min(t.heads, G - hb * t.heads);
    it.seen = s.n - s.nq + i0 + 1;
    it.n = s.n;
    const int32_t last = max(0, it.seen + it.toks - 1), tiles = (last + BN - 1) / BN;
    // tiles in equal parts, the first ones with one more where they do not divide
    const int32_t each = quotient(tiles, parts), more = tiles - each * parts;
    it.tiles = each + (p < more ? 1 : 0);
    it.k0 = (p * each + min(p, more)) * BN;
    it.part = parts > 1 ? part0 + x : -1;
    it.box = it.toks <= t.few ? t.few : t.tok;
    it.b = b;
    it.hk = hk;
    return true;
}

// ------------------------------------------------------------------ parts of a row, joined

// O = sum_p 2^(L_p - m) O_p / sum_p 2^(L_p - m), L_p the part's log-sum-exp in base 2: in one pass with a running
// maximum, a few parts at a time, all of their loads before the first use. LANES lanes hold a row, each VECS pieces
// of four dims, 4 LANES dims apart.
template <int VECS, int LANES>
struct Joined {
    static constexpr int AT_ONCE = VECS > 4 ? 2 : 4;
    float m, l;
    float4 o[VECS];
    __device__ __forceinline__ void add(int x, float w, const float4& y) {
        o[x] = make_float4(fmaf(w, y.x, o[x].x), fmaf(w, y.y, o[x].y), fmaf(w, y.z, o[x].z), fmaf(w, y.w, o[x].w));
    }
    __device__ __forceinline__ float weight(float lse) const { return ex2(lse - (m == -INFINITY ? 0.f : m)); }
    __device__ __forceinline__ void rescale(float to) {  // to a maximum of at least m
        const float f = m == to ? 1.f : ex2(m - to);
        l *= f;
#pragma unroll
        for (int x = 0; x < VECS; ++x) o[x] = make_float4(o[x].x * f, o[x].y * f, o[x].z * f, o[x].w * f);
        m = to;
    }
    // Parts p = from, from + by, .. below n; mine: this lane's first piece of part 0, lses: the row's sum of part 0.
    // Plain loads: the parts are the kernel before's, visible since grid_wait.
    __device__ __forceinline__ void parts(const float* mine, const float* lses, int64_t step, int from, int by, int n, int lane,
                                          int D) {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int x = 0; x < VECS; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int32_t p0 = from; p0 < n; p0 += AT_ONCE * by) {
            float lse[AT_ONCE];
            float4 y[AT_ONCE][VECS];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int32_t p = p0 + i * by;
                lse[i] = p < n ? lses[p * step] : -INFINITY;
#pragma unroll
                for (int x = 0; x < VECS; ++x)
                    y[i][x] = p < n && 4 * (lane + LANES * x) < D
                                  ? *reinterpret_cast<const float4*>(mine + p * step + 4 * LANES * x)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) top = fmaxf(top, lse[i]);
            rescale(top);
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const float w = weight(lse[i]);
                l += w;
#pragma unroll
                for (int x = 0; x < VECS; ++x) add(x, w, y[i][x]);
            }
        }
    }
    __device__ __forceinline__ void write(__nv_bfloat16* dst, float* lse, int lane, int D) const {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int x = 0; x < VECS; ++x)
            if (4 * (lane + LANES * x) < D)
                *reinterpret_cast<uint2*>(dst + 4 * LANES * x) =
                    make_uint2(pack_bf16(o[x].x * inv, o[x].y * inv), pack_bf16(o[x].z * inv, o[x].w * inv));
        if (lane == 0) *lse = l == 0.f ? -INFINITY : (m + lg2(l)) * kLn2;
    }
};

// ------------------------------------------------------------------ the tile kernel

template <int D>
struct Layout {
    static constexpr int BN = block_n(D), KVS = stages(D), CH = D / 64;
    static constexpr int TILE_Q = kTile * D * 2;
    static constexpr int TILE_KV = BN * D * 2;
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = Q_OFF + TILE_Q;
    static constexpr int V_OFF = K_OFF + KVS * TILE_KV;
    static constexpr int BAR_OFF = V_OFF + KVS * TILE_KV;
    static constexpr int B_QFULL = 0, B_QEMPTY = 1;
    static constexpr int B_KFULL = 2, B_KEMPTY = B_KFULL + KVS;
    static constexpr int B_VFULL = B_KEMPTY + KVS, B_VEMPTY = B_VFULL + KVS, B_VFIX = B_VEMPTY + KVS;
    static constexpr int B_SFULL = B_VFIX + KVS;               // 2
    static constexpr int B_PFULL = B_SFULL + 2;                // 2
    static constexpr int B_ODONE = B_PFULL + 2;
    static constexpr int B_OFREE = B_ODONE + 1;
    static constexpr int B_OFULL = B_OFREE + 1;                // last product of an item complete
    static constexpr int B_DRAIN = B_OFULL + 1;
    static constexpr int B_RFULL = B_DRAIN + 1, B_REMPTY = B_RFULL + 2;   // items: 2 slots
    static constexpr int NBAR = B_REMPTY + 2;
    static constexpr int ITEM_OFF = BAR_OFF + (NBAR * 8 + 15) / 16 * 16;
    static constexpr int MISC_OFF = ITEM_OFF + 2 * (int)sizeof(Item);   // TMEM base, abort flag, 4 x item with values to add
    static constexpr int BYTES = MISC_OFF + 32;
    static constexpr size_t ALLOC = (size_t)BYTES + 1024;      // slack for 1024-byte alignment
};

// Whether any of the eight bf16 of x is not finite: x - x is zero or NaN.
__device__ __forceinline__ bool not_finite8(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
        const __nv_bfloat162 d = __hsub2(v, v);
        any |= *reinterpret_cast<const uint32_t*>(&d);
    }
    return any != 0;
}

// Those replaced by zeros.
__device__ __noinline__ uint4 only_finite(uint4 x) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
        if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0x0000ffffu;
    }
    return x;
}

// 32 bytes to global memory, 32-byte aligned: a whole sector of a row that one lane writes.
__device__ __forceinline__ void store32(void* to, const uint32_t* x) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// 16 bytes of global memory to shared memory, or zeros, asynchronously.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
                 "r"(there ? 16 : 0)
                 : "memory");
}
// An arrival on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }

// What the table holds for slot j of an item's sequence, kNone behind the last.
constexpr int32_t kNone = INT32_MIN;
__device__ __forceinline__ int32_t entry_of(const PagedAttendArgs& a, int32_t b, int32_t n, int64_t j) {
    return j < n ? max(a.table[(int64_t)b * a.table_ld + (j >> a.c.shift)], -1) : kNone;
}
// The page that it names; `pages`, which holds nothing, for none and for one outside the pool.
__device__ __forceinline__ int32_t page_of(const PagedAttendArgs& a, int32_t entry) {
    if ((uint32_t)entry < (uint32_t)a.c.pages) return entry;
    if (entry != kNone) set_error(a.status, ATTN_E_BOUNDS);
    return a.c.pages;
}

// Sum of V's values in dim d of slots [from, to) that are not finite: those that the products left
// out, because other rows of the tile do not see them.
__device__ __noinline__ float not_finite(const PagedAttendArgs& a, int32_t b, int32_t hk, int32_t n, int32_t from,
                                         int32_t to, int d) {
    float sum = 0.f;
    for (int32_t j = from; j < to && d < a.g.D; ++j) {
        const int32_t id = page_of(a, entry_of(a, b, n, j));
        if (id >= a.c.pages) continue;
        const uint32_t v = static_cast<const uint16_t*>(a.c.v)[id * a.c.sp + hk * a.c.sh +
                                                                (j & ((1 << a.c.shift) - 1)) * a.c.st + d];
        if ((v & 0x7f80u) == 0x7f80u) sum += __uint_as_float(v << 16);
    }
    return sum;
}

template <int D, bool GATHER>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmq_few,
                  const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const __grid_constant__ PagedAttendArgs a, const TcMaps mpq, const TcMaps mpkv,
                  const __grid_constant__ Tiling t) {
    using LY = Layout<D>;
    constexpr int BN = LY::BN, KVS = LY::KVS, CH = LY::CH;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(sm);
    const uint32_t bar0 = sbase + LY::BAR_OFF;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    Item* slot = reinterpret_cast<Item*>(sm + LY::ITEM_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + LY::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + LY::MISC_OFF + 4);
    volatile uint32_t* to_add = reinterpret_cast<volatile uint32_t*>(sm + LY::MISC_OFF + 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(bar(LY::B_QFULL), 1);
        mbar_init(bar(LY::B_QEMPTY), 1);
        for (int s = 0; s < KVS; ++s) {
            mbar_init(bar(LY::B_KFULL + s), 1);
            mbar_init(bar(LY::B_KEMPTY + s), 1);
            mbar_init(bar(LY::B_VFULL + s), GATHER ? 64 : 1);       // every lane of warps 2 and 3
            mbar_init(bar(LY::B_VEMPTY + s), 1);
            mbar_init(bar(LY::B_VFIX + s), 2);         // warps 2 and 3
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(LY::B_SFULL + s), 1);
            mbar_init(bar(LY::B_PFULL + s), 128);
            mbar_init(bar(LY::B_RFULL + s), 1);
            mbar_init(bar(LY::B_REMPTY + s), 7);       // MMA thread, warps 2 and 3, 4 softmax warps
        }
        mbar_init(bar(LY::B_ODONE), 1);
        mbar_init(bar(LY::B_OFREE), 128);
        mbar_init(bar(LY::B_OFULL), 1);
        mbar_init(bar(LY::B_DRAIN), 1);
        *abort_flag = 0;
        for (int i = 0; i < 4; ++i) to_add[i] = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    if (tid == 32) {
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmq_few);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_wait();
    grid_go();
    const uint32_t tmem = *tmem_slot;

    // the next item, for a consumer that is one thread or a warp (`one`: this lane arrives for it)
    auto next_item = [&](uint32_t ic, Item& it, bool one) {
        const uint32_t s = ic & 1;
        if (!mbar_wait(bar(LY::B_RFULL + s), (ic >> 1) & 1, abort_flag, a.status, a.wait_ns)) return false;
        const volatile int32_t* p = reinterpret_cast<const volatile int32_t*>(slot + s);
        int32_t* to = reinterpret_cast<int32_t*>(&it);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Item) / 4); ++i) to[i] = p[i];
        if (one) mbar_arrive(bar(LY::B_REMPTY + s));
        return it.tiles >= 0 && !*abort_flag;
    };
    auto next_item_warp = [&](uint32_t ic, Item& it) {
        const bool go = __all_sync(0xffffffffu, next_item(ic, it, false));
        if (lane == 0) mbar_arrive(bar(LY::B_REMPTY + (ic & 1)));
        return go;
    };

    const int boxes = BN / t.box;                       // of a tile
    const int window = 32 / boxes;                      // tiles whose pages a warp's lanes hold
    const int box_shift = 31 - __clz(t.box);
    // table entry of box `lane` of an item's tiles from `first` on
    auto pages_at = [&](const Item& it, int32_t first) {
        const int64_t j = (int64_t)it.k0 + (int64_t)first * BN + lane * t.box;
        return lane < window * boxes && first < it.tiles ? entry_of(a, it.b, it.n, j) : kNone;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ items and loads
        const List L = make_list<BN>(a, t, blockIdx.x == 0);
        Found at{-1, 0, 0, 0};
        // item w of the list and its first table entries
        auto look_up = [&](int32_t w, Item& it, int32_t& entries) {
            it.tiles = -1;
            entries = kNone;
            if (w >= L.n_items) return;
            if (find_item<BN>(a, t, L, at, w, it)) {
                entries = pages_at(it, 0);
            } else {
                it.tiles = -1;
                if (lane == 0) {
                    set_error(a.status, ATTN_E_BOUNDS);
                    *abort_flag = 1;
                }
            }
        };
        auto claim = [&]() {
            int32_t w = 0;
            if (lane == 0) w = (int32_t)min(atomicAdd(a.counter, 1u) + gridDim.x, (uint32_t)INT32_MAX);
            return __shfl_sync(0xffffffffu, w, 0);
        };
        uint32_t kc = 0, ne = 0;
        Item it{}, next{};
        int32_t ahead = kNone, ahead_next = kNone;
        bool ok = !a.stall;
        if (ok) look_up((int32_t)blockIdx.x, it, ahead);
        for (uint32_t ic = 0; ok; ++ic) {
            ok = mbar_wait_warp(bar(LY::B_REMPTY + (ic & 1)), ((ic >> 1) & 1) ^ 1, abort_flag, a.status, a.wait_ns);
            if (!ok) break;
            if (lane == 0) {
                volatile int32_t* p = reinterpret_cast<volatile int32_t*>(slot + (ic & 1));
                const int32_t* from = reinterpret_cast<const int32_t*>(&it);
#pragma unroll
                for (int i = 0; i < (int)(sizeof(Item) / 4); ++i) p[i] = from[i];
                mbar_arrive(bar(LY::B_RFULL + (ic & 1)));
            }
            __syncwarp();
            if (it.tiles < 0 || __any_sync(0xffffffffu, *abort_flag)) break;
            if (it.tiles > 0) {
                ok = mbar_wait_warp(bar(LY::B_QEMPTY), (ne & 1) ^ 1, abort_flag, a.status, a.wait_ns);
                if (!ok) break;
                const bool few = it.box == t.few && t.few < t.tok;
                if (lane == 0) mbar_expect_tx(bar(LY::B_QFULL), (uint32_t)(it.box * t.heads * 128 * CH));
                __syncwarp();
                if (lane < CH) {
                    const int c1 = mpq.pos_t == 1 ? it.tok0 : (mpq.pos_h == 1 ? it.head0 : 0);
                    const int c2 = mpq.pos_t == 2 ? it.tok0 : (mpq.pos_h == 2 ? it.head0 : 0);
                    const int c3 = mpq.pos_t == 3 ? it.tok0 : (mpq.pos_h == 3 ? it.head0 : 0);
                    tma_load_4d(sbase + LY::Q_OFF + lane * (kTile * 128), few ? &tmq_few : &tmq, bar(LY::B_QFULL),
                                lane * 64, c1, c2, c3);
                }
                ++ne;
                // one lane a box: 64 dims of the slots of a page (or of a tile, if pages are longer)
                const int bi = lane / CH, bc = lane - bi * CH;
                const bool loads = lane < boxes * CH;
                int32_t now = 0;
                for (int32_t j = 0; j < it.tiles && ok; ++j) {
                    const int32_t in = j % window;
                    if (in == 0) {
                        now = page_of(a, ahead);
                        ahead = pages_at(it, j + window);
                    }
                    const int32_t id = __shfl_sync(0xffffffffu, now, (in * boxes + bi) & 31);
                    const int32_t place = (it.k0 + j * BN + bi * t.box) & ((1 << a.c.shift) - 1);
                    const int c1 = mpkv.pos_t == 1 ? place : (mpkv.pos_h == 1 ? it.hk : id);
                    const int c2 = mpkv.pos_t == 2 ? place : (mpkv.pos_h == 2 ? it.hk : id);
                    const int c3 = mpkv.pos_t == 3 ? place : (mpkv.pos_h == 3 ? it.hk : id);
                    const uint32_t s = kc % KVS, turn = (kc / KVS) & 1;
                    const uint32_t off = s * LY::TILE_KV + bc * (BN * 128) + bi * t.box * 128;
                    ok = mbar_wait_warp(bar(LY::B_KEMPTY + s), turn ^ 1, abort_flag, a.status, a.wait_ns);
                    if (!ok) break;
                    if (lane == 0) mbar_expect_tx(bar(LY::B_KFULL + s), LY::TILE_KV);
                    __syncwarp();
                    if (loads) tma_load_4d(sbase + LY::K_OFF + off, &tmk, bar(LY::B_KFULL + s), bc * 64, c1, c2, c3);
                    if (!GATHER) {
                        ok = mbar_wait_warp(bar(LY::B_VEMPTY + s), turn ^ 1, abort_flag, a.status, a.wait_ns);
                        if (!ok) break;
                        if (lane == 0) mbar_expect_tx(bar(LY::B_VFULL + s), LY::TILE_KV);
                        __syncwarp();
                        if (loads) tma_load_4d(sbase + LY::V_OFF + off, &tmv, bar(LY::B_VFULL + s), bc * 64, c1, c2, c3);
                    }
                    ++kc;
                    // the next item is looked up while the last tile loads (four tiles earlier: 512 sequences of 3000
                    // slots at most 471 us against 467, chunks of four prompts 193 and 190; sixteen: 478 and 192)
                    if (j == it.tiles - 1) look_up(claim(), next, ahead_next);
                }
                if (!ok) break;
            } else {
                look_up(claim(), next, ahead_next);
            }
            it = next;
            ahead = ahead_next;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (elect_one()) {
            constexpr uint32_t id_s = idesc_bf16(128, BN, 0, 0);
            constexpr uint32_t id_o = idesc_bf16(128, D, 0, 1);
            uint32_t kc = 0, ne = 0, gt = 0;            // gt: tiles so far (S buffer, P, product)
            Item it;
            bool ok = true;
            for (uint32_t ic = 0; ok; ++ic) {
                if (!next_item(ic, it, true)) break;
                if (it.tiles == 0) continue;
                ok = mbar_wait(bar(LY::B_QFULL), ne & 1, abort_flag, a.status, a.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t q0 = sbase + LY::Q_OFF;
                uint32_t vc = kc;
                for (int j = 0; j <= it.tiles && ok; ++j) {
                    if (j < it.tiles) {
                        const uint32_t ks = kc % KVS;
                        ok = mbar_wait(bar(LY::B_KFULL + ks), (kc / KVS) & 1, abort_flag, a.status, a.wait_ns);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t k0 = sbase + LY::K_OFF + ks * LY::TILE_KV;
                        const uint32_t sb = tmem + kColS + ((gt + j) & 1) * BN;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t qoff = (kk >> 2) * (kTile * 128) + (kk & 3) * 32;
                            const uint32_t koff = (kk >> 2) * (BN * 128) + (kk & 3) * 32;
                            mma_ss(sb, sdesc_sw128(q0 + qoff, 16, 1024), sdesc_sw128(k0 + koff, 16, 1024), id_s, kk > 0);
                        }
                        mma_commit(bar(LY::B_KEMPTY + ks));
                        mma_commit(bar(LY::B_SFULL + ((gt + j) & 1)));
                        ++kc;
                        if (j == it.tiles - 1) mma_commit(bar(LY::B_QEMPTY));
                    }
                    if (j >= 1) {
                        const uint32_t x = gt + j - 1, pb = x & 1;
                        if (j == 1) {
                            ok = mbar_wait(bar(LY::B_OFREE), (ne & 1) ^ 1, abort_flag, a.status, a.wait_ns);
                            if (!ok) break;
                        }
                        const uint32_t vs = vc % KVS;
                        ok = mbar_wait(bar(LY::B_VFULL + vs), (vc / KVS) & 1, abort_flag, a.status, a.wait_ns) &&
                             (GATHER ||
                              mbar_wait(bar(LY::B_VFIX + vs), (vc / KVS) & 1, abort_flag, a.status, a.wait_ns)) &&
                             mbar_wait(bar(LY::B_PFULL + pb), (x >> 1) & 1, abort_flag, a.status, a.wait_ns);
                        if (!ok) break;
                        if (GATHER) fence_proxy_async_smem();      // V came by copies of the generic proxy
                        tc_fence_after();
                        const uint32_t v0 = sbase + LY::V_OFF + vs * LY::TILE_KV;
                        const uint32_t pa = tmem + kColS + pb * BN;
#pragma unroll
                        for (int kk = 0; kk < BN / 16; ++kk)
                            mma_ts(tmem + kColO, pa + kk * 8, sdesc_sw128(v0 + kk * 2048, BN * 128, 1024), id_o,
                                   (j - 1 > 0 || kk > 0) ? 1u : 0u);
                        mma_commit(bar(LY::B_VEMPTY + vs));
                        mma_commit(bar(LY::B_ODONE));
                        if (j == it.tiles) mma_commit(bar(LY::B_OFULL));
                        ++vc;
                    }
                }
                gt += it.tiles;
                ++ne;
            }
        }
    } else if (warp < 4 && GATHER) {
        // ------------------------------------------------------------ V by 16-byte copies, half a tile each
        constexpr int PIECES = D / 8, ROWS = 32 / PIECES, STEPS = 16 / ROWS;   // of a row; rows a step; steps of 16 rows
        constexpr int BLOCKS = BN / 32;                  // of 16 rows, in a warp's half of a tile
        const int piece = lane % PIECES, r_lane = lane / PIECES;
        const bool in_row = piece * 8 < a.g.D;
        // this lane's place in a tile: rows r_lane + ROWS i, whose low bits the swizzle mixes into the piece's
        const uint32_t ring = sbase + LY::V_OFF + (piece >> 3) * (BN * 128) + r_lane * 128;
        const uint32_t mixed = (uint32_t)((piece & 7) ^ r_lane);
        const __nv_bfloat16* rows = static_cast<const __nv_bfloat16*>(a.c.v) + (in_row ? piece * 8 : 0);
        const int64_t step = ROWS * a.c.st;
        Item it;
        bool ok = true;
        uint32_t kc = 0, ne = 0;
        for (uint32_t ic = 0; ok; ++ic) {
            if (!next_item_warp(ic, it)) break;
            if (it.tiles == 0) continue;
            int32_t ahead = pages_at(it, 0), now = 0;
            const __nv_bfloat16* head = rows + it.hk * a.c.sh;
            for (int32_t j = 0; j < it.tiles; ++j) {
                const int32_t in = j % window;
                if (in == 0) {
                    now = page_of(a, ahead);
                    ahead = pages_at(it, j + window);
                }
                // the addresses first, while the stage may still be read
                const int32_t j0 = it.k0 + j * BN + (warp - 2) * (BN / 2);   // this warp's half
                const __nv_bfloat16* src[BLOCKS];
                int32_t used[BLOCKS];                    // rows from this lane's first on that hold a slot in use
#pragma unroll
                for (int x = 0; x < BLOCKS; ++x) {
                    const int32_t id = __shfl_sync(
                        0xffffffffu, now, (in * boxes + (((warp - 2) * (BN / 2) + x * 16) >> box_shift)) & 31);
                    const int32_t first = j0 + x * 16 + r_lane;
                    const bool page = in_row && id < a.c.pages;
                    src[x] = page ? head + id * a.c.sp + (first & ((1 << a.c.shift) - 1)) * a.c.st : rows;
                    used[x] = page ? it.n - first : 0;
                }
                const uint32_t s = kc % KVS;
                ok = mbar_wait_warp(bar(LY::B_VEMPTY + s), ((kc / KVS) & 1) ^ 1, abort_flag, a.status, a.wait_ns);
                if (!ok) break;
                const uint32_t dst = ring + s * LY::TILE_KV + (warp - 2) * (BN / 2) * 128;
                const bool some = j0 + BN / 2 > it.seen && it.seen < it.n;   // some rows are not seen by all
                if (!some) {
#pragma unroll
                    for (int x = 0; x < BLOCKS; ++x)
#pragma unroll
                        for (int i = 0; i < STEPS; ++i)
                            copy16(dst + (x * 16 + i * ROWS) * 128 + ((mixed ^ ((i * ROWS) & 7)) << 4), src[x] + i * step,
                                   i * ROWS < used[x]);
                    copy_arrive(bar(LY::B_VFULL + s));
                } else {
                    bool any = false;
#pragma unroll 1
                    for (int x = 0; x < BLOCKS; ++x) {
                        const int32_t all = it.seen - (j0 + x * 16 + r_lane);      // rows before it are seen by all
                        const __nv_bfloat16* from = src[0];
                        int32_t rows_used = used[0];
#pragma unroll
                        for (int y = 1; y < BLOCKS; ++y)
                            if (x == y) {
                                from = src[y];
                                rows_used = used[y];
                            }
                        uint4 v[STEPS];
#pragma unroll
                        for (int i = 0; i < STEPS; ++i)
                            v[i] = i * ROWS < rows_used ? *reinterpret_cast<const uint4*>(from + i * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < STEPS; ++i) {
                            if (i * ROWS >= all && not_finite8(v[i])) {
                                v[i] = only_finite(v[i]);
                                any = true;
                            }
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(
                                             dst + (x * 16 + i * ROWS) * 128 + ((mixed ^ ((i * ROWS) & 7)) << 4)),
                                         "r"(v[i].x), "r"(v[i].y), "r"(v[i].z), "r"(v[i].w)
                                         : "memory");
                        }
                    }
                    if (any) to_add[ne & 3] = ne + 1;
                    mbar_arrive(bar(LY::B_VFULL + s));
                }
                ++kc;
            }
            ++ne;
        }
        copy_wait_all();
    } else if (warp < 4) {
        // ------------------------------------------------------------ what no row may see of V
        Item it;
        bool ok = true;
        uint32_t vc = 0, ne = 0;
        for (uint32_t ic = 0; ok; ++ic) {
            if (!next_item_warp(ic, it)) break;
            if (it.tiles == 0) continue;
            for (int j = 0; j < it.tiles && ok; ++j, ++vc) {
                const uint32_t vs = vc % KVS;
                ok = mbar_wait_warp(bar(LY::B_VFULL + vs), (vc / KVS) & 1, abort_flag, a.status, a.wait_ns);
                if (!ok) break;
                const int32_t j0 = it.k0 + j * BN;
                if (j0 + BN > it.seen) {
                    const int r0 = max(0, it.seen - j0), rn = min(max(it.n - j0, 0), BN);   // rows [rn, BN) hold no slot in use
                    uint8_t* v = sm + LY::V_OFF + vs * LY::TILE_KV;
                    bool any = false;
                    // 16-byte pieces of 64 dims of a row: eight lanes a row, four rows a warp, eight steps in flight
                    constexpr int AT_ONCE = 8 / CH;
#pragma unroll 1
                    for (int y = r0 + (warp - 2) * 4 + (lane >> 3); y < BN; y += 8 * AT_ONCE) {
                        uint4 x[AT_ONCE][CH];
#pragma unroll
                        for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
                            for (int c = 0; c < CH; ++c)
                                if (y + 8 * i < rn)
                                    x[i][c] = *reinterpret_cast<const uint4*>(v + c * (BN * 128) + (y + 8 * i) * 128 + (lane & 7) * 16);
#pragma unroll
                        for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
                            for (int c = 0; c < CH; ++c) {
                                uint4* p = reinterpret_cast<uint4*>(v + c * (BN * 128) + (y + 8 * i) * 128 + (lane & 7) * 16);
                                if (y + 8 * i < rn) {
                                    if (not_finite8(x[i][c])) {
                                        *p = only_finite(x[i][c]);
                                        any = true;
                                    }
                                } else if (y + 8 * i < BN) {
                                    *p = make_uint4(0, 0, 0, 0);
                                }
                            }
                    }
                    if (any) to_add[ne & 3] = ne + 1;
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(LY::B_VFIX + vs));
            }
            ++ne;
        }
    } else {
        // ------------------------------------------------------------ softmax / epilogue
        const int row = tid - 128;                       // TMEM lane == tile row
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const float sl2 = a.g.scale * kLog2e;
        uint32_t gt = 0, ne = 0;
        bool ok = true;
        Item it;
        for (uint32_t ic = 0; ok; ++ic) {
            if (!next_item_warp(ic, it)) break;
            // this row's token and head
            const int maj = t.head_major ? it.box : t.heads, hi = row / maj, lo = row - hi * maj;
            const int ti = t.head_major ? lo : hi, gi = t.head_major ? hi : lo;
            const bool live = ti < it.toks && gi < it.heads;
            const uint32_t rows = __ballot_sync(0xffffffffu, live);
            const bool warp_live = rows != 0;
            const float lag = __popc(rows) <= kExactRows ? 0.f : kLag;
            const int32_t seen = it.seen + ti;           // slots [0, seen)
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = 0; j < it.tiles && ok; ++j) {
                const uint32_t x = gt + j, b = x & 1;
                ok = mbar_wait_warp(bar(LY::B_SFULL + b), (x >> 1) & 1, abort_flag, a.status, a.wait_ns);
                if (!ok) break;
                if (!warp_live) {                        // rows that nobody reads
                    mbar_arrive(bar(LY::B_PFULL + b));
                    continue;
                }
                tc_fence_after();
                constexpr int NC = BN / 32;
                const uint32_t sa = tmem + lane_addr + kColS + b * BN;
                uint32_t r[NC][32];
#pragma unroll
                for (int c = 0; c < NC; ++c) tmem_ld32(sa + c * 32, r[c]);
                tmem_ld_wait();
                const int j0 = it.k0 + j * BN;
                float mul = sl2;
                if (j0 + BN > it.seen || !(sl2 > 0.f)) {
                    // scaled before they are masked and compared, whatever the scale's sign
                    const int lim = seen - j0;           // columns c < lim are seen
                    mul = 1.f;
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            r[c][i] = __float_as_uint((c * 32 + i < lim) ? __uint_as_float(r[c][i]) * sl2 : -INFINITY);
                }
                float hi4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        hi4[(c * 2 + (i >> 4)) & 3] =
                            fmax3(hi4[(c * 2 + (i >> 4)) & 3], __uint_as_float(r[c][i]), __uint_as_float(r[c][i + 1]));
                const float mt = fmax3(fmaxf(hi4[0], hi4[1]), hi4[2], hi4[3]) * mul;
                bool rescale = false;
                float alpha = 1.f;
                if (mt > m_run + lag) {
                    if (m_run != -INFINITY) {
                        rescale = true;
                        alpha = ex2(m_run - mt);
                    }
                    m_run = mt;
                }
                const float base = m_run == -INFINITY ? 0.f : m_run;
                const float2 mul2 = make_float2(mul, mul), nbase = make_float2(-base, -base);
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t p[NC / 2][32];
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 e =
                            ffma2(make_float2(__uint_as_float(r[c][i]), __uint_as_float(r[c][i + 1])), mul2, nbase);
                        const float p0 = ex2(e.x), p1 = ex2(e.y);
                        acc[(i >> 1) & 1] = fadd2(acc[(i >> 1) & 1], make_float2(p0, p1));
                        p[c >> 1][(c & 1) * 16 + (i >> 1)] = pack_bf16(p0, p1);
                    }
                const float lsum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                l_run = rescale ? fmaf(l_run, alpha, lsum) : l_run + lsum;
#pragma unroll
                for (int c2 = 0; c2 < NC / 2; ++c2) tmem_st32(sa + 32 * c2, p[c2]);
                if (__any_sync(0xffffffffu, rescale) && j > 0) {
                    // O holds the sum over the item's earlier tiles once their products have completed
                    ok = mbar_wait_warp(bar(LY::B_ODONE), (x - 1) & 1, abort_flag, a.status, a.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t oa = tmem + lane_addr + kColO;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(oa + c * 32, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(oa + c * 32, o);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(LY::B_PFULL + b));
            }
            if (!ok) break;
            const int Dv = a.g.D, tok = it.tok0 + ti, h = it.head0 + gi;
            const bool empty = it.tiles == 0;
            bool add = false;
            if (!empty) {
                ok = mbar_wait_warp(bar(LY::B_OFULL), ne & 1, abort_flag, a.status, a.wait_ns);
                if (!ok) break;
                tc_fence_after();
                add = to_add[ne & 3] == ne + 1;
            }
            // values to add: the slots of this item's tiles that not all of its rows see
            const int32_t add0 = max(max(it.seen, 0), it.k0), add1 = min(seen, it.k0 + it.tiles * BN);
            const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
            const float lse2 = l_run == 0.f ? -INFINITY : m_run + lg2(l_run);
            const uint32_t oa = tmem + lane_addr + kColO;
            if (warp_live) {
                __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.o) + (int64_t)tok * a.g.st + (int64_t)h * a.g.sh;
                const int at = ti * t.heads + gi;
                float* base = a.parts + it.part * t.part_floats;
                float* part = base + (int64_t)at * Dv;
                if (live) {
                    if (it.part < 0)
                        a.lse[(int64_t)h * a.g.T + tok] = lse2 * kLn2;
                    else
                        base[(int64_t)t.part_rows * Dv + at] = lse2;
                }
                // as much of O at a time as the scores took registers
                constexpr int AT_ONCE = BN / 32;
#pragma unroll
                for (int c0 = 0; c0 < D / 32; c0 += AT_ONCE) {
                    uint32_t o[AT_ONCE][32];
#pragma unroll
                    for (int c = 0; c < AT_ONCE; ++c) {
                        if (c0 + c >= D / 32) break;
                        if (!empty) {
                            tmem_ld32(oa + (c0 + c) * 32, o[c]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[c][i] = 0;
                        }
                    }
                    tmem_ld_wait();
                    if (!live) continue;
#pragma unroll
                    for (int c = 0; c < AT_ONCE; ++c) {
                        const int d0 = (c0 + c) * 32;
                        if (d0 >= D) break;
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[c][i] = __float_as_uint(__uint_as_float(o[c][i]) * inv);
                        if (it.part < 0) {
                            uint32_t y[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                y[i] = pack_bf16(__uint_as_float(o[c][2 * i]), __uint_as_float(o[c][2 * i + 1]));
#pragma unroll
                            for (int i = 0; i < 16; i += 8) {
                                if (d0 + 2 * i >= Dv) break;
                                if (t.wide) {
                                    store32(dst + d0 + 2 * i, y + i);
                                } else {
                                    *reinterpret_cast<uint4*>(dst + d0 + 2 * i) = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                                    if (d0 + 2 * i + 8 < Dv)
                                        *reinterpret_cast<uint4*>(dst + d0 + 2 * i + 8) =
                                            make_uint4(y[i + 4], y[i + 5], y[i + 6], y[i + 7]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 8)
                                if (d0 + i < Dv)
                                    store32(part + d0 + i, &o[c][i]);
                        }
                    }
                }
                if (add && live) {
#pragma unroll 1
                    for (int d = 0; d < Dv; ++d) {
                        const float x = not_finite(a, it.b, it.hk, it.n, add0, add1, d);
                        if (x == 0.f) continue;
                        if (it.part < 0)
                            dst[d] = __float2bfloat16(__bfloat162float(dst[d]) + x);
                        else
                            part[d] += x;
                    }
                }
            }
            if (empty) continue;
            tc_fence_before();
            mbar_arrive(bar(LY::B_OFREE));
            gt += it.tiles;
            ++ne;
        }
    }
    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        if (*abort_flag) {
            // a wait gave up: let the MMAs already issued drain (bounded) before TMEM is released
            if (elect_one()) {
                mma_commit(bar(LY::B_DRAIN));
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(bar(LY::B_DRAIN), 0) && globaltimer() - t0 < a.wait_ns) {
                }
            }
            __syncwarp();
        }
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ parts of cut units, joined

constexpr int kMergeWarps = 8;

// The last sequence that begins at or before the token.
__device__ __forceinline__ int32_t sequence_at(const int32_t* cu, int32_t B, int32_t tok) {
    int32_t b = 0;
    for (int32_t hi = B; hi - b > 1;) {
        const int32_t mid = (b + hi) >> 1;
        if (cu[mid] <= tok) b = mid; else hi = mid;
    }
    return b;
}

// By the offsets that the kernel before put in order; out of line, which keeps the join's registers free.
__device__ __noinline__ int32_t sequence_taken(const PagedAttendArgs& a, int32_t tok) { return sequence_at(a.offsets, a.B, tok); }

// LPR lanes a row of the output: the whole block up to 8 rows an SM, a warp up to 64, a quarter of a warp beyond. Chunks of
// 32 heads over 32K slots, by block, warp and quarter: 32 rows 34.0, 37.7 and 50.4 us, 640 rows 36.8, 39.8 and 55.0, 1216
// rows (8 an SM) 45.2, 44.1 and 51.0, 2432 rows 58.7, 54.5 and 59.2; 9728 rows (64 an SM) 185, 163 and 167, 19456 rows 228,
// 210.5 and 209, chunks of four prompts (97K rows and more) 309, 202 and 192. Row r is head r % H of token r / H. Also leaves the work queue at zero for the next call.
template <int LPR, int DT>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const PagedAttendArgs a, const Tiling t) {
    constexpr int ROWS = 32 * kMergeWarps / LPR;
    constexpr bool BLOCK = ROWS == 1;                    // the block's warps take parts in turn
    constexpr int LANES = BLOCK ? 32 : LPR;              // over a row's dims
    constexpr int VECS = DT / 4 / LANES;                 // float4 of a row that a lane holds
    __shared__ float red[2][kMergeWarps];
    __shared__ __align__(16) float sums[BLOCK ? kMergeWarps : 1][BLOCK ? DT : 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x % LANES, sub = BLOCK ? warp : 0, subs = BLOCK ? kMergeWarps : 1;
    const int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR;
    // the row's sequence, tokens [q0, to): offsets are older than the kernel before this one
    const bool there = r < (int64_t)a.g.T * a.g.H;       // the same for the lanes of a row
    const int32_t tok = there ? (int32_t)((uint32_t)r / (uint32_t)a.g.H) : 0, h = (int32_t)(r - (int64_t)tok * a.g.H);
    int32_t b, q0, to;
    if (a.cu) {
        b = sequence_at(a.cu, a.B, tok);
        q0 = a.cu[b];
        to = a.cu[b + 1];
    } else {
        b = min(tok / a.each, a.B - 1);
        q0 = b * a.each;
        to = q0 + a.each;
    }
    grid_wait();
    grid_go();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.counter = 0;
    if (!there) return;
    int4 cut = a.cuts[b];
    if (cut.w) {                                         // offsets out of order: as the kernel before took them
        b = sequence_taken(a, tok);
        q0 = a.offsets[b];
        to = a.offsets[b + 1];
        cut = a.cuts[b];
    }
    if (cut.y <= 1 || tok < q0 || tok >= to) return;
    const int32_t row_tiles = row_tiles_of(t, to - q0), hk = h / t.group, g = h - hk * t.group;
    const int32_t hb = g / t.heads, i = tok - q0, rt = (int32_t)t.by_tok.div((uint32_t)i);
    const int32_t row = (i - rt * t.tok) * t.heads + (g - hb * t.heads);
    // part p of this row is partial first + p * apart; units in front of cut.z are whole
    const int32_t unit = (hk * t.blocks + hb) * row_tiles + (row_tiles - 1 - rt), apart = cut.z ? t.units * row_tiles - cut.z : row_tiles;
    if (unit < cut.z) return;
    const int64_t first = cut.x + (cut.z ? unit - cut.z : (int64_t)(hk * t.blocks + hb) * cut.y * row_tiles + (row_tiles - 1 - rt));
    if (first + (int64_t)(cut.y - 1) * apart >= a.max_parts || row >= t.part_rows) {
        if (lane == 0) set_error(a.status, ATTN_E_BOUNDS);
        return;
    }
    const float* base = a.parts + first * t.part_floats;
    const int64_t step = (int64_t)apart * t.part_floats;
    const int32_t D = a.g.D;
    const float* lses = base + (int64_t)t.part_rows * D + row;
    Joined<VECS, LANES> j;
    j.parts(base + (int64_t)row * D + 4 * lane, lses, step, sub, subs, cut.y, lane, D);
    if (BLOCK) {
        if (lane == 0) {
            red[0][warp] = j.m;
            red[1][warp] = j.l;
        }
#pragma unroll
        for (int x = 0; x < VECS; ++x) *reinterpret_cast<float4*>(&sums[warp][4 * (lane + LANES * x)]) = j.o[x];
        __syncthreads();
        if (warp != 0) return;
        float top = j.m;
        for (int w = 1; w < kMergeWarps; ++w) top = fmaxf(top, red[0][w]);
        j.rescale(top);
        for (int w = 1; w < kMergeWarps; ++w) {
            const float f = j.weight(red[0][w]);
            j.l = fmaf(f, red[1][w], j.l);
#pragma unroll
            for (int x = 0; x < VECS; ++x) j.add(x, f, *reinterpret_cast<const float4*>(&sums[w][4 * (lane + LANES * x)]));
        }
    }
    j.write(reinterpret_cast<__nv_bfloat16*>(a.o) + (int64_t)tok * a.g.st + (int64_t)h * a.g.sh + 4 * lane,
            a.lse + (int64_t)h * a.g.T + tok, lane, D);
}

template <int D, bool GATHER>
cudaError_t launch_d(const PagedAttendArgs& a, cudaStream_t s) {
    CUtensorMap mq, mq_few, mk, mv;
    TcMaps mpq{1, 2, 3}, mpkv{1, 2, 3};
    Tiling t = tiling(a.c, a.g);
    const Geom kv = a.c.geom();
    if (!make_tile_map(&mq, a.q, a.g, mpq, t.tok, t.heads) || !make_tile_map(&mq_few, a.q, a.g, mpq, t.few, t.heads) ||
        !make_tile_map(&mk, a.c.k, kv, mpkv, t.box) || !make_tile_map(&mv, a.c.v, kv, mpkv, t.box))
        return cudaErrorInvalidValue;
    t.head_major = mpq.pos_t < mpq.pos_h;
    t.wide = ((uintptr_t)a.o | (uintptr_t)(2 * a.g.st) | (uintptr_t)(2 * a.g.sh) | (uintptr_t)(2 * a.g.D)) % 32 == 0;
    static_assert(Layout<D>::ALLOC <= 232448, "shared memory of the paged attention's kernel");
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, GATHER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Layout<D>::ALLOC);
    if (e != cudaSuccess) return e;
    e = launch_early(attend_kernel<D, GATHER>, dim3(device_sm_count()), kThreads, Layout<D>::ALLOC, 1, s, mq, mq_few, mk, mv, a,
                     mpq, mpkv, t);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)a.g.T * a.g.H;
    constexpr int kBlock = 32 * kMergeWarps, DT = D < 128 ? 128 : D;
    auto merge = [&](auto kernel, int lanes) {
        const int64_t per = kBlock / lanes;
        return launch_early(kernel, dim3((unsigned)((rows + per - 1) / per)), kBlock, 0, 1, s, a, t);
    };
    if (rows <= 8 * t.sms) return merge(merge_kernel<kBlock, DT>, kBlock);
    return rows <= 64 * t.sms ? merge(merge_kernel<32, DT>, 32) : merge(merge_kernel<8, DT>, 8);
}

}  // namespace

size_t paged_parts_bytes(const PagedGeom& c, const Geom& g, int32_t* max_parts) {
    // a unit of n tiles that is cut has at most 2 n / C parts, and C is at least the work of an SM / kItemsPerSm,
    // up to a rounding of fp32
    const Tiling t = tiling(c, g);
    *max_parts = (2 * kItemsPerSm + 1) * t.sms;
    return (size_t)*max_parts * t.part_floats * sizeof(float);
}

bool paged_units_fit(const PagedGeom& c, const Geom& g, int64_t B) {
    const Tiling t = tiling(c, g);
    return ((int64_t)g.T / t.tok + B) * c.Hkv * t.blocks <= (1 << 30);
}

cudaError_t launch_paged_attend(const PagedAttendArgs& a, cudaStream_t s) {
    // head dims run on tiles of 64, 128 or 256, as the forward's
    const bool gather = a.c.page() <= kGatherPage;
    if (a.g.D > 128) return gather ? launch_d<256, true>(a, s) : launch_d<256, false>(a, s);
    if (a.g.D > 64) return gather ? launch_d<128, true>(a, s) : launch_d<128, false>(a, s);
    return gather ? launch_d<64, true>(a, s) : launch_d<64, false>(a, s);
}

}  // namespace attn
